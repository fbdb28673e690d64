"""Plain 64-bit implementations of the operators around the recurrent branch
(the formulas of include/gdn.h), in numpy on the host, and the error bounds of
the library's arithmetic against them."""
from __future__ import annotations

import numpy as np
import torch

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def stored_sum(x, residual):
    """x + residual in binary32, rounded to the residual's type (x alone
    without one), as a CPU tensor."""
    if residual is None:
        return x.cpu()
    return (x.cpu().float() + residual.cpu().float()).to(residual.dtype)


def codes(g):
    """Codes and largest magnitude of each row of g (binary64)."""
    with np.errstate(all="ignore"):
        top = np.abs(g).max(-1)
        top = np.where(np.isfinite(g).all(-1), top, np.nan)
        q = np.rint(127.0 * g / top[:, None])
        q[~np.isfinite(q)] = 0
    return q.astype(np.int8), top


def rmsnorm_q8(h, w, eps):
    """Codes and binary64 scales of the rows h (stored values) with weight w."""
    h, w = f64(h), f64(w)
    with np.errstate(all="ignore"):
        q, top = codes(h * w)
        scale = top / 127.0 / np.sqrt((h * h).mean(-1) + float(np.float32(eps)))
    scale[top == 0] = 0.0
    return q, scale


def quantize_q8(x):
    q, top = codes(f64(x))
    return q, top / 127.0


def linear_q8(a, a_scale, w, w_scale, bias, dtype):
    """y in binary64 and the bound of the library's error: the 32-bit integer
    sum is exact; its conversion, the two scalings (each half a binary32 step
    of the scaled sum) and the bias (half a step of the result) come before one
    rounding to the output's type.  fp16 also rounds to its smallest step,
    2^-24, near zero."""
    acc = f64(a) @ f64(w).T                       # exact: below 2^53
    s = acc * f64(a_scale)[:, None] * f64(w_scale)
    y = s + (f64(bias) if bias is not None else 0.0)
    u = 2.0 ** -24
    tol = 3 * u * np.abs(s) * (1 + 4 * u) + u * np.abs(y)
    tol = tol + (np.abs(y) + tol) * (torch.finfo(dtype).eps / 2)
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    return y, tol + 1e-38


def weights(p):
    p = np.asarray(p, np.float64)
    return np.where((p > 0) & np.isfinite(p), p, 0.0)


def verify(target, draft, draft_tokens, u_accept, u_sample, n_draft=None):
    """accepted [B] and tokens [B][K+1], position by position."""
    t = f64(target)
    q = None if draft is None else f64(draft)
    d = draft_tokens.cpu().numpy()
    ua, us = f64(u_accept), f64(u_sample)
    B, K1, V = t.shape
    K = K1 - 1
    n = np.full(B, K) if n_draft is None else np.clip(n_draft.cpu().numpy(), 0, K)
    accepted = np.zeros(B, np.int32)
    tokens = np.full((B, K1), -1, np.int32)
    for b in range(B):
        a, refused = 0, False
        while a < n[b]:
            tok = d[b, a]
            ok = False
            if 0 <= tok < V:
                pd = weights(t[b, a, tok])
                qd = 1.0 if q is None else weights(q[b, a, tok])
                ok = bool(ua[b, a] * qd < pd)
            if not ok:
                refused = True
                break
            tokens[b, a] = tok
            a += 1
        p = weights(t[b, a])
        rest = p
        if refused:
            if q is None:
                one = np.zeros(V)
                if 0 <= d[b, a] < V:
                    one[d[b, a]] = 1.0
                rest = np.maximum(p - one, 0.0)
            else:
                rest = np.maximum(p - weights(q[b, a]), 0.0)
        w = rest if rest.sum() > 0 else p
        cum = np.cumsum(w)
        hit = np.nonzero((cum > us[b] * w.sum()) & (w > 0))[0]
        live = np.nonzero(w > 0)[0]
        tokens[b, a] = hit[0] if len(hit) else (live[-1] if len(live) else -1)
        accepted[b] = a
    return accepted, tokens
