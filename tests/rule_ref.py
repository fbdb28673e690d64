"""The delta rule over packed sequences in 64 bits on the host: the recurrence
token by token, its gradient by the adjoint recurrence, and the bounds of the
library's arithmetic against them."""
from __future__ import annotations

import torch

D = 128
CHUNK = 64
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def inputs(lens, hv, hk, dtype, seed, tail=0, start=True, gate=None, pool=None, device="cuda"):
    """Packed tokens of sequences of the given lengths, `tail` rows behind the
    last, states in a pool of `pool` slots (None: one a sequence)."""
    gen = torch.Generator().manual_seed(seed)
    n = max(1, sum(lens) + tail)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    unit = torch.nn.functional.normalize
    x = dict(q=unit(rnd(n, hk, D), dim=-1).to(dtype), k=unit(rnd(n, hk, D), dim=-1).to(dtype),
             v=rnd(n, hv, D).to(dtype), beta=torch.sigmoid(rnd(n, hv)),
             gate=-torch.nn.functional.softplus(rnd(n, hv)) if gate is None else torch.full((n, hv), float(gate)))
    starts = [0]
    for m in lens:
        starts.append(starts[-1] + m)
    x["offsets"] = torch.tensor(starts, dtype=torch.int32)
    x["slots"] = None
    if pool is not None:
        x["slots"] = torch.randperm(pool, generator=gen)[:len(lens)].to(torch.int32)
    x["state"] = 0.1 * rnd(pool or len(lens), hv, D, D) if start else None
    x["d_out"] = rnd(n, hv, D).to(dtype)
    x["d_state_out"] = 0.1 * rnd(len(lens), hv, D, D)
    return {a: None if t is None else t.to(device) for a, t in x.items()}


def _host(x):
    return {a: None if t is None else t.detach().cpu().double() if t.is_floating_point() else t.cpu()
            for a, t in x.items()}


def _spans(x):
    o, n = x["offsets"].tolist(), x["q"].shape[0]
    spans, slots = [], x["slots"].tolist() if x["slots"] is not None else list(range(len(o) - 1))
    for b in range(len(o) - 1):
        first = max(0, min(o[b], n))
        spans.append((first, max(first, max(0, min(o[b + 1], n))), slots[b]))
    return spans


def forward(x):
    """out, state_out (the given pool with the sequences' states replaced), and
    for each output the size of what is summed for it: the norm of the row that
    enters its chunk and the magnitudes of the chunk's corrections, over sqrt(128).
    The states' is returned alike, without the root and over all chunks."""
    x = _host(x)
    n, hv = x["v"].shape[:2]
    heads = torch.arange(hv) % x["q"].shape[1]
    out, size = torch.zeros(n, hv, D, dtype=torch.float64), torch.zeros(n, hv, D, dtype=torch.float64)
    spans = _spans(x)
    slots = x["state"].shape[0] if x["state"] is not None else len(spans)
    pool = x["state"].clone() if x["state"] is not None else torch.zeros(slots, hv, D, D, dtype=torch.float64)
    psize = torch.zeros(slots, hv, D, 1, dtype=torch.float64)
    for first, end, slot in spans:
        if not 0 <= slot < slots:
            continue
        m = pool[slot].clone()
        top = m.norm(dim=-1)
        for c in range(first, end, CHUNK):
            entered, total = m.norm(dim=-1), torch.zeros(hv, D, dtype=torch.float64)
            stop = min(end, c + CHUNK)
            for t in range(c, stop):
                k, q = x["k"][t, heads], x["q"][t, heads]
                m = torch.exp(x["gate"][t])[:, None, None] * m
                delta = x["beta"][t][:, None] * (x["v"][t] - (m @ k[..., None])[..., 0])
                m = m + delta[..., None] * k[:, None]
                out[t] = (m @ q[..., None])[..., 0] / D ** 0.5
                total += delta.abs()
            size[c:stop] = (entered + total) / D ** 0.5
            top = top + entered + total
        pool[slot] = m
        psize[slot] = top[..., None]
    return out, pool, size, psize


def backward(x):
    """Gradients of sum(out * d_out) + sum(state_out * d_state_out); rows of no
    sequence get zeros."""
    x = _host(x)
    n, hv = x["v"].shape[:2]
    hk = x["q"].shape[1]
    heads = torch.arange(hv) % hk
    z = {a: torch.zeros(x[a].shape[0], hv, *x[a].shape[2:], dtype=torch.float64) for a in ("q", "k", "v", "beta", "gate")}
    ds = torch.zeros(len(_spans(x)), hv, D, D, dtype=torch.float64)
    for b, (first, end, slot) in enumerate(_spans(x)):
        m = x["state"][slot].clone() if x["state"] is not None else torch.zeros(hv, D, D, dtype=torch.float64)
        path = []
        for t in range(first, end):
            k = x["k"][t, heads]
            kept = torch.exp(x["gate"][t])[:, None, None] * m
            miss = x["v"][t] - (kept @ k[..., None])[..., 0]
            m = kept + (x["beta"][t][:, None] * miss)[..., None] * k[:, None]
            path.append((kept, miss, m))
        g = x["d_state_out"][b].clone() if x["d_state_out"] is not None else torch.zeros(hv, D, D, dtype=torch.float64)
        for t in reversed(range(first, end)):
            kept, miss, after = path[t - first]
            k, q, do = x["k"][t, heads], x["q"][t, heads], x["d_out"][t] / D ** 0.5
            z["q"][t] = (do[:, None] @ after)[:, 0]
            g = g + do[..., None] * q[:, None]
            dd = (g @ k[..., None])[..., 0]
            z["beta"][t] = (dd * miss).sum(-1)
            dm = x["beta"][t][:, None] * dd
            z["v"][t] = dm
            z["k"][t] = ((x["beta"][t][:, None] * miss)[:, None] @ g)[:, 0] - (dm[:, None] @ kept)[:, 0]
            g = g - dm[..., None] * k[:, None]
            z["gate"][t] = (g * kept).sum((-1, -2))
            g = torch.exp(x["gate"][t])[:, None, None] * g
        ds[b] = g
    share = lambda y: y.unflatten(1, (hv // hk, hk)).sum(1)
    return dict(dq=share(z["q"]), dk=share(z["k"]), dv=z["v"], dbeta=z["beta"], dgate=z["gate"], d_state=ds)


def out_bound(y, size, dtype):
    """gdn_chunk's outputs: 16-bit ones are rounded once (half a step, and half
    the smallest step of fp16) from sums whose operands are cut at 2^-16 twice, so
    2^-15 of the terms, and as much again for what the corrections carry; float32
    ones come of at most 192 binary32 sums of terms right to 2^-23."""
    if dtype == torch.float32:
        return 200 * 2.0 ** -24 * size * 2 + 1e-30
    half = torch.finfo(dtype).eps / 2
    return half * y.abs() + 2.0 ** -14 * size * (1 + half) + (2.0 ** -25 if dtype == torch.float16 else 0) + 1e-30


def state_bound(size):
    """192 binary32 sums a chunk of terms right to 2^-23, over all chunks (size
    adds them up), twice for what a chunk's corrections carry on."""
    return 2 * 200 * 2.0 ** -24 * size + 1e-30


def rel(a, b):
    b = b.double()
    return float((a.detach().cpu().double() - b).norm() / (b.norm() + 1e-300))
