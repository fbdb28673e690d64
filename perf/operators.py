"""Cases of the operators around the recurrent step: the quantised norm, the
8-bit projections, the verification of drafted tokens and the commit of a
speculative pair.  Each case can be run in a plain form (elementary torch
operations) or through the library (`own`)."""
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
D = 128            # head size of the recurrent state
RING = 3           # slots of the conv ring
ACCEPTED = 0.7     # how often a drafted token of prepare() is about accepted


def listed():
    return [
        # one decoded token entering a layer: the hidden width of the page's geometry
        dict(name="norm_row1_n2048", op="norm", rows=1, n=2048, x="f32", res="f32"),
        # 8 prompts x 4096 tokens entering a layer
        dict(name="norm_row32768_n2048", op="norm", rows=32768, n=2048, x="bf16", res="bf16"),
        # the tail's y of 32 decoded tokens before the output projection
        dict(name="quant_row32_n4096", op="quant", rows=32, n=4096, x="f32"),
        # the same over a packed batch of prompts, with an odd width
        dict(name="quant_row20001_n4097", op="quant", rows=20001, n=4097, x="bf16"),
        # one decoded token through the three input projections of a layer
        dict(name="linear_m1_in", op="linear", m=1, k=2048, n0=8192, n1=4096, n2=64, out="f32", bias=False),
        # a ragged handful of tokens, odd in every size
        dict(name="linear_m77_odd", op="linear", m=77, k=1111, n0=1003, n1=0, n2=0, out="f16", bias=True),
        # 256 decoded tokens through the output projection
        dict(name="linear_m256_out", op="linear", m=256, k=4096, n0=2048, n1=0, n2=0, out="f32", bias=False),
        # 8 prompts x 4096 tokens through the three input projections
        dict(name="linear_m32768_in", op="linear", m=32768, k=2048, n0=8192, n1=4096, n2=64, out="bf16", bias=False),
        # one sequence, one drafted token (the pair), a small vocabulary
        dict(name="verify_b1_v32000", op="verify", b=1, drafts=1, v=32000, probs="f32", greedy=False, ragged=False),
        # a large batch with up to three drafts each, a large odd vocabulary
        dict(name="verify_b256_v131071", op="verify", b=256, drafts=3, v=131071, probs="bf16", greedy=False, ragged=True),
        # one sequence's speculative pair in one layer
        dict(name="commit_b1", op="commit", layers=1, b=1, heads=32, channels=8192),
        # a decode batch of 256 sequences in one layer
        dict(name="commit_b256", op="commit", layers=1, b=256, heads=32, channels=8192),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "quant", "linear", "linear", "verify", "commit"])
    kinds = ["f32", "bf16", "f16"]
    if op in ("norm", "quant"):
        n = _log_int(rng, 1, 20000)
        rows = _log_int(rng, 1, max(2, min(100000, (1 << 25) // n)))
        c = dict(op=op, rows=rows, n=n, x=rng.choice(kinds))
        return dict(c, res=rng.choice(kinds + ["none"])) if op == "norm" else c
    if op == "linear":
        k = _log_int(rng, 1, 16384)
        n0 = _log_int(rng, 1, 16384)
        n1 = rng.choice([0, 0, _log_int(rng, 1, 4096)])
        n2 = rng.choice([0, _log_int(rng, 1, 128)]) if n1 else 0
        if rng.random() < 0.6:      # widths are whole vectors more often than not
            k, n0 = (k + 63) // 64 * 64, (n0 + 15) // 16 * 16
        most = int(5e11 / (k * (n0 + n1 + n2)))
        m = _log_int(rng, 1, max(2, min(16384, most)))
        return dict(op=op, m=m, k=k, n0=n0, n1=n1, n2=n2, out=rng.choice(kinds), bias=rng.random() < 0.3)
    if op == "verify":
        v = _log_int(rng, 1000, 262144)
        drafts = rng.randint(1, 8)
        b = _log_int(rng, 1, max(2, min(256, (1 << 27) // (v * (2 * drafts + 1)))))
        return dict(op=op, b=b, drafts=drafts, v=v, probs=rng.choice(kinds), greedy=rng.random() < 0.3,
                    ragged=rng.random() < 0.5)
    layers = rng.randint(1, 4)
    heads = rng.choice([16, 32, 48, 64])
    b = _log_int(rng, 1, max(2, 256 * 32 // (heads * layers)))
    return dict(op="commit", layers=layers, b=b, heads=heads, channels=rng.choice([0, 4 * D * heads // 2]))


def _outs(c):
    return [n for n in (c["n0"], c["n1"], c["n2"]) if n]


def _library():
    import gated_deltanet_decode_amd as gdn
    return gdn


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, dev = case, "cuda"

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, device=dev, generator=gen) * std).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, device=dev, generator=gen)

    s = {"case": c}
    if c["op"] in ("norm", "quant"):
        s["x"] = normal(c["rows"], c["n"], dtype=TYPES[c["x"]])
        s["q"] = torch.empty(c["rows"], c["n"], dtype=torch.int8, device=dev)
        s["scale"] = torch.empty(c["rows"], device=dev)
        if c["op"] == "norm":
            s["w"] = 1.0 + normal(c["n"], std=0.02)
            s["residual"] = s["residual_out"] = None
            if c["res"] != "none":
                # the residual stream, summed up over earlier layers
                s["residual"] = normal(c["rows"], c["n"], std=3.0, dtype=TYPES[c["res"]])
                s["residual_out"] = torch.empty_like(s["residual"])
    elif c["op"] == "linear":
        total = sum(_outs(c))
        s["a"] = normal(c["m"], c["k"], std=32.0).round_().clamp_(-127, 127).to(torch.int8)
        s["w"] = normal(total, c["k"], std=32.0).round_().clamp_(-127, 127).to(torch.int8)
        s["a_scale"] = 0.01 + 0.04 * uniform(c["m"])
        s["w_scale"] = 0.0002 + 0.001 * uniform(total)
        s["bias"] = normal(total) if c["bias"] else None
        s["outs"] = [torch.empty(c["m"], n, dtype=TYPES[c["out"]], device=dev) for n in _outs(c)]
    elif c["op"] == "verify":
        b, k, v, t = c["b"], c["drafts"], c["v"], TYPES[c["probs"]]
        s["target"] = torch.empty(b, k + 1, v, dtype=t, device=dev)
        s["draft"] = None if c["greedy"] else torch.empty(b, k, v, dtype=t, device=dev)
        s["tokens_in"] = torch.empty(b, k, dtype=torch.int32, device=dev)
        for i in range(k + 1):
            logits = normal(b, v, std=2.5)
            s["target"][:, i] = torch.softmax(logits, -1)
            if i < k:
                q = torch.softmax(logits + normal(b, v, std=0.8), -1)
                s["tokens_in"][:, i] = torch.multinomial(q, 1, generator=gen)[:, 0] if not c["greedy"] else q.argmax(-1)
                if not c["greedy"]:
                    s["draft"][:, i] = q
        s["n_draft"] = None
        if c["ragged"]:
            s["n_draft"] = torch.randint(0, k + 1, (b,), device=dev, generator=gen, dtype=torch.int32)
        s["u_accept"], s["u_sample"] = uniform(b, k), uniform(b)
        s["accepted"] = torch.empty(b, dtype=torch.int32, device=dev)
        s["tokens"] = torch.empty(b, k + 1, dtype=torch.int32, device=dev)
        if own:
            # the scratch a caller keeps from step to step
            s["ws"] = torch.empty(_library().verify_workspace_bytes(b, v), dtype=torch.uint8, device=dev)
    else:
        shape = (c["layers"], c["b"], c["heads"], D, D)
        s["state"], s["state_next"] = normal(*shape, std=0.1), normal(*shape, std=0.1)
        s["ring"] = s["ring_next"] = None
        if c["channels"]:
            ring = (c["layers"], c["b"], RING, c["channels"])
            s["ring"], s["ring_next"] = normal(*ring), normal(*ring)
        s["accepted"] = (uniform(c["b"]) < ACCEPTED).to(torch.int32)
        if c["b"] == 1:
            s["accepted"].fill_(1)
    return s


def _quantised(g):
    """Codes in [-127, 127] of the rows of g (64 bits) and each row's largest
    magnitude; 64 bits, since a code that falls next to a border has to be the same
    however the row was summed."""
    top = g.abs().amax(-1, keepdim=True)
    codes = torch.round(127.0 * g / top)
    return torch.where(torch.isfinite(codes), codes, torch.zeros_like(codes)), top


def _weights(p):
    return torch.where((p > 0) & torch.isfinite(p), p, torch.zeros_like(p))


def _plain_verify(s):
    c = s["case"]
    b, k, v = c["b"], c["drafts"], c["v"]
    dev = s["target"].device
    d = s["tokens_in"].long()
    at = torch.arange(k, device=dev)
    n = s["n_draft"].long() if s["n_draft"] is not None else torch.full((b,), k, device=dev)
    p_d = _weights(s["target"][:, :k].gather(2, d[:, :, None])[:, :, 0].double())
    q_d = torch.ones_like(p_d) if s["draft"] is None else _weights(s["draft"].gather(2, d[:, :, None])[:, :, 0].double())
    good = (s["u_accept"].double() * q_d < p_d) & (at[None] < n[:, None])
    a = good.long().cumprod(1).sum(1)
    refused = a < n
    i = torch.arange(b, device=dev)
    p = _weights(s["target"][i, a].double())
    pos = torch.clamp(a, max=k - 1)
    if s["draft"] is None:
        q = torch.zeros_like(p).scatter_(1, d[i, pos][:, None], 1.0)
    else:
        q = _weights(s["draft"][i, pos].double())
    rest = torch.clamp(p - q * refused[:, None], min=0.0)
    w = torch.where((rest.sum(1) > 0)[:, None], rest, p)
    cum = w.cumsum(1)
    hit = (cum > s["u_sample"].double()[:, None] * w.sum(1, keepdim=True)) & (w > 0)
    ids = torch.arange(v, device=dev)[None]
    first = torch.where(hit, ids, v).amin(1)
    last = torch.where(w > 0, ids, -1).amax(1)
    token = torch.where(first < v, first, last)
    cols = torch.arange(k + 1, device=dev)[None]
    padded = torch.cat([d, d[:, :1]], 1)
    tokens = torch.where(cols < a[:, None], padded, torch.where(cols == a[:, None], token[:, None], -1))
    return {"accepted": a.int(), "tokens": tokens.int()}


def run(state):
    s, c = state, state["case"]
    if c["op"] == "norm":
        if own:
            _library().add_rmsnorm_q8(s["x"], s["residual"], s["residual_out"], s["w"], s["q"], s["scale"], eps=EPS)
            h, scale = s["residual_out"], s["scale"]
            values = s["q"] * scale[:, None]
        else:
            h = None
            base = s["x"]
            if s["residual"] is not None:
                h = base = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
            wide = base.double()
            q, top = _quantised(wide * s["w"].double())
            rms = torch.sqrt(wide.square().mean(-1, keepdim=True) + EPS)
            scale = (top / 127.0 / rms)[:, 0].float()
            values = q.float() * scale[:, None]
        out = {"values": values, "scale": scale}
        return dict(out, residual=h) if h is not None else out
    if c["op"] == "quant":
        if own:
            _library().quantize_q8(s["x"], s["q"], s["scale"])
            return {"values": s["q"] * s["scale"][:, None], "scale": s["scale"]}
        q, top = _quantised(s["x"].double())
        scale = (top / 127.0)[:, 0].float()
        return {"values": q.float() * scale[:, None], "scale": scale}
    if c["op"] == "linear":
        if own:
            _library().linear_q8(s["a"], s["a_scale"], s["w"], s["w_scale"], s["outs"], bias=s["bias"])
            return s["outs"]
        y = (s["a"].float() @ s["w"].float().t()) * s["a_scale"][:, None] * s["w_scale"]
        if s["bias"] is not None:
            y = y + s["bias"]
        return [p.to(TYPES[c["out"]]) for p in y.split(_outs(c), 1)]
    if c["op"] == "verify":
        if own:
            _library().verify(s["target"], s["draft"], s["tokens_in"], s["u_accept"], s["u_sample"], s["accepted"],
                              s["tokens"], n_draft=s["n_draft"], workspace=s["ws"])
            return {"accepted": s["accepted"], "tokens": s["tokens"]}
        return _plain_verify(s)
    if own:
        _library().pair_commit(s["accepted"], s["state"], s["state_next"], s["ring"], s["ring_next"])
        return [s["state"]] + ([s["ring"]] if s["ring"] is not None else [])
    keep = s["accepted"] > 0
    out = [torch.where(keep[None, :, None, None, None], s["state_next"], s["state"])]
    if s["ring"] is not None:
        out.append(torch.where(keep[None, :, None, None], s["ring_next"], s["ring"]))
    return out


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits; the verification's
    whole numbers have no such value."""
    c = case
    if c["op"] == "verify":
        return None
    s = prepare(case, seed)
    if c["op"] == "commit":
        took = s["accepted"].nonzero()[:, 0]
        out = []
        for now, later in (("state", "state_next"), ("ring", "ring_next")):
            if s[now] is not None:
                out.append(s[now].double())
                out[-1][:, took] = s[later][:, took].double()
        return out
    if c["op"] == "linear":
        y = torch.matmul(s["a"].double(), s["w"].double().t().contiguous())
        y = y.mul_(s["w_scale"].double()).mul_(s["a_scale"].double()[:, None])
        if s["bias"] is not None:
            y += s["bias"].double()
        return list(torch.split(y, _outs(c), 1))
    h, out = s["x"].double(), {}
    if c["op"] == "norm":
        if s["residual"] is not None:
            h = h + s["residual"].double()
            out["residual"] = h
            # the norm is taken of the stored sum
            h = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype).double()
        normed = h * s["w"].double()
        size = torch.sqrt((h * h).sum(-1) / c["n"] + EPS)
    else:
        normed, size = h, torch.ones(c["rows"], dtype=torch.float64, device=h.device)
    top = torch.max(normed.abs(), -1).values
    step = top / 127.0
    codes = (127.0 * normed / top[:, None]).round()
    codes[top == 0] = 0
    out["scale"] = step / size
    out["values"] = codes * (step / size)[:, None]
    return out


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "f16": 2, "none": 0}
    if c["op"] in ("norm", "quant"):
        e = c["rows"] * c["n"]
        b = e * (size[c["x"]] + 1) + 4 * c["rows"]
        if c["op"] == "norm":
            b += 2 * e * size[c["res"]] + 4 * c["n"]
        return {"bytes": b, "flops": 6 * e}
    if c["op"] == "linear":
        n = sum(_outs(c))
        b = (c["m"] + n) * (c["k"] + 4) + c["m"] * n * size[c["out"]] + (4 * n if c["bias"] else 0)
        return {"bytes": b, "flops": 2 * c["m"] * n * c["k"]}
    if c["op"] == "verify":
        # one target row a sequence, and the draft's row where a token was refused
        refused = 0.5 if c["ragged"] else 1 - ACCEPTED ** c["drafts"]
        rows = c["b"] * (1 + (0 if c["greedy"] else refused))
        return {"bytes": rows * c["v"] * size[c["probs"]] + 8 * c["b"] * (c["drafts"] + 1), "flops": 3 * rows * c["v"]}
    share = 1 if c["b"] == 1 else ACCEPTED
    floats = c["layers"] * c["b"] * (c["heads"] * D * D + RING * c["channels"])
    return {"bytes": 8 * share * floats, "flops": 0}
