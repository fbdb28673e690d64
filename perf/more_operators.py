"""Cases of the gated delta rule in chunks (forward, backward, and its form for
single tokens), the products in 8-bit floating point with a scale for each block
of 128, and the log probabilities of answered tokens.  Each case can be run in a
plain form (elementary torch operations) or through the library (`own`)."""
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
F8 = torch.float8_e4m3fn
F8_MOST = 448.0
BLOCK = 128        # elements that share a scale
D = 128            # head size of the recurrent state
C = 64             # tokens of a chunk in the plain form
SCALE = D ** -0.5  # of the read-out


def listed():
    return [
        # one short prompt through the recurrent branch, starting from no state
        dict(name="chunk_b1_t200", op="chunk", b=1, t=200, ragged=False, hv=32, hk=16, type="bf16", start=False),
        # 8 prompts x 4096 tokens
        dict(name="chunk_b8_t4096", op="chunk", b=8, t=4096, ragged=False, hv=32, hk=16, type="bf16", start=True),
        # the gradient of one short training sequence
        dict(name="backward_b1_t333", op="backward", b=1, t=333, ragged=False, hv=32, hk=16, type="bf16", start=False),
        # the gradient of a training batch of packed sequences of up to 4096 tokens
        dict(name="backward_b8_t4096", op="backward", b=8, t=4096, ragged=True, hv=32, hk=16, type="bf16", start=True),
        # one decoded token of one sequence
        dict(name="decode_b1", op="decode", b=1, t=1, ragged=False, hv=32, hk=16, type="bf16", pool=4),
        # a decode batch of 256 sequences whose states lie anywhere in a pool
        dict(name="decode_b256", op="decode", b=256, t=1, ragged=False, hv=32, hk=16, type="bf16", pool=300),
        # the tail's y of 32 decoded tokens before the output projection
        dict(name="quant_f8_row32_n4096", op="quant", rows=32, n=4096, x="f32", block_rows=1),
        # 8 prompts x 4096 tokens entering a layer
        dict(name="quant_f8_row32768_n2048", op="quant", rows=32768, n=2048, x="bf16", block_rows=1),
        # one decoded token through the three input projections of a layer
        dict(name="linear_f8_m1_in", op="linear", m=1, k=2048, n0=8192, n1=4096, n2=64, out="f32", bias=False),
        # 8 prompts x 4096 tokens through the three input projections
        dict(name="linear_f8_m32768_in", op="linear", m=32768, k=2048, n0=8192, n1=4096, n2=64, out="bf16", bias=False),
        # the answer of two sequences' decode step, a small vocabulary
        dict(name="logprobs_r2_v32000", op="logprobs", rows=2, v=32000, logits="f32", top=5),
        # 256 sequences with three drafts each, a large odd vocabulary
        dict(name="logprobs_r1024_v131071", op="logprobs", rows=1024, v=131071, logits="bf16", top=20),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "backward", "backward", "decode", "quant", "linear", "linear", "logprobs"])
    kinds = ["f32", "bf16", "f16"]
    if op in ("chunk", "backward"):
        hv, hk = rng.choice([(32, 16), (32, 32), (16, 4), (48, 16), (5, 5)])
        t = _log_int(rng, 1, 8192)
        b = _log_int(rng, 1, max(2, min(64, 8 * 4096 * 32 // (hv * t * 2))))
        return dict(op=op, b=b, t=t, ragged=rng.random() < 0.6, hv=hv, hk=hk,
                    type=rng.choice(["bf16", "bf16", "f16", "f32"]), start=rng.random() < 0.5)
    if op == "decode":
        hv, hk = rng.choice([(32, 16), (32, 32), (16, 4), (48, 16)])
        b = _log_int(rng, 1, 256 * 32 // hv)
        return dict(op=op, b=b, t=rng.choice([1, 1, 1, 2, 4, 7]), ragged=rng.random() < 0.4, hv=hv, hk=hk,
                    type=rng.choice(kinds), pool=b + rng.randint(0, 20))
    if op == "quant":
        n = _log_int(rng, 1, 20000)
        rows = _log_int(rng, 1, max(2, min(100000, (1 << 26) // n)))
        return dict(op=op, rows=rows, n=n, x=rng.choice(kinds), block_rows=rng.choice([1, 1, BLOCK]))
    if op == "linear":
        k = _log_int(rng, 1, 16384)
        n0 = _log_int(rng, 1, 16384)
        n1 = rng.choice([0, 0, _log_int(rng, 1, 4096)])
        n2 = rng.choice([0, _log_int(rng, 1, 128)]) if n1 else 0
        if rng.random() < 0.6:      # widths are whole blocks more often than not
            k, n0 = (k + 127) // 128 * 128, (n0 + 15) // 16 * 16
        most = int(5e11 / (k * (n0 + n1 + n2)))
        m = _log_int(rng, 1, max(2, min(16384, most)))
        return dict(op=op, m=m, k=k, n0=n0, n1=n1, n2=n2, out=rng.choice(kinds), bias=rng.random() < 0.3)
    v = _log_int(rng, 1000, 262144)
    rows = _log_int(rng, 1, max(2, min(1024, (1 << 27) // v)))
    return dict(op=op, rows=rows, v=v, logits=rng.choice(kinds), top=rng.choice([0, 1, 5, 20, 32]))


def _lens(c):
    """Tokens of each sequence, t at most: where ragged, spread over [0, t] by a
    sequence that fills the range evenly, the first of them whole."""
    if not c["ragged"]:
        return [c["t"]] * c["b"]
    return [round(c["t"] * (1 - i * 0.6180339887498949 % 1)) for i in range(c["b"])]


def _outs(c):
    return [n for n in (c["n0"], c["n1"], c["n2"]) if n]


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _library():
    import gated_deltanet_decode_amd as gdn
    return gdn


def _prepare_rule(s, c, normal, uniform):
    """Packed tokens of all sequences, and a few rows behind the last."""
    lens, t = _lens(c), TYPES[c["type"]]
    n = sum(lens) + (3 if c["ragged"] else 0)
    n = max(n, 1)
    hv, hk = c["hv"], c["hk"]
    starts = [0]
    for m in lens:
        starts.append(starts[-1] + m)
    s["lens"] = lens
    s["offsets"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    unit = torch.nn.functional.normalize
    s["q"] = unit(normal(n, hk, D), dim=-1).to(t)
    s["k"] = unit(normal(n, hk, D), dim=-1).to(t)
    s["v"] = normal(n, hv, D, dtype=t)
    s["beta"] = torch.sigmoid(normal(n, hv))
    # log decays of trained heads: from slow to fast ones
    rate = torch.exp(-5.0 + 6.0 * uniform(hv))
    s["gate"] = -rate * torch.nn.functional.softplus(normal(n, hv))
    if c["op"] == "decode":
        perm = torch.argsort(uniform(c["pool"]))[:c["b"]]
        s["slots"] = perm.to(torch.int32)
        s["state"] = normal(c["pool"], hv, D, D, std=0.1)
        s["state_out"] = s["state"].clone()
    else:
        s["slots"] = None
        s["state"] = normal(c["b"], hv, D, D, std=0.1) if c["start"] else None
        s["state_out"] = torch.zeros(c["b"], hv, D, D, device="cuda")
    if c["op"] == "backward":
        s["d_out"] = normal(n, hv, D, dtype=t)
        # what a next segment of the sequence hands back
        s["d_state_out"] = normal(c["b"], hv, D, D, std=0.1) if c["start"] else None
        s["d_state"] = torch.empty(c["b"], hv, D, D, device="cuda") if c["start"] else None
        for name in ("q", "k", "v", "beta", "gate"):
            s["d" + name] = torch.zeros_like(s[name])
    else:
        s["out"] = torch.zeros(n, hv, D, dtype=t, device="cuda")
    if own and c["op"] != "decode":
        gdn = _library()
        size = gdn.chunk_workspace_bytes if c["op"] == "chunk" else gdn.chunk_backward_workspace_bytes
        # the scratch a caller keeps from call to call
        s["ws"] = torch.empty(size(c["b"], n, t, gdn.Dims(hv, hk, D, D)), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, dev = case, "cuda"

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, device=dev, generator=gen) * std).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, device=dev, generator=gen)

    s = {"case": c}
    if c["op"] in ("chunk", "backward", "decode"):
        _prepare_rule(s, c, normal, uniform)
    elif c["op"] == "quant":
        s["x"] = normal(c["rows"], c["n"], dtype=TYPES[c["x"]])
        s["q"] = torch.empty(c["rows"], c["n"], dtype=F8, device=dev)
        tall = c["rows"] if c["block_rows"] == 1 else _blocks(c["rows"])
        s["scale"] = torch.empty(tall, _blocks(c["n"]), device=dev)
    elif c["op"] == "linear":
        total = sum(_outs(c))
        s["a"] = normal(c["m"], c["k"], std=100.0).clamp_(-F8_MOST, F8_MOST).to(F8)
        s["w"] = normal(total, c["k"], std=100.0).clamp_(-F8_MOST, F8_MOST).to(F8)
        s["a_scale"] = 0.003 + 0.01 * uniform(c["m"], _blocks(c["k"]))
        s["w_scale"] = 0.0001 + 0.0003 * uniform(_blocks(total), _blocks(c["k"]))
        s["bias"] = normal(total) if c["bias"] else None
        s["outs"] = [torch.empty(c["m"], n, dtype=TYPES[c["out"]], device=dev) for n in _outs(c)]
    else:
        r, v = c["rows"], c["v"]
        s["logits"] = normal(r, v, std=2.5, dtype=TYPES[c["logits"]])
        # a twentieth of the vocabulary masked, as a grammar leaves it
        s["logits"][:, torch.nonzero(uniform(v) < 0.05)[:, 0]] = float("-inf")
        near = s["logits"].float() + normal(r, v)      # another sampler's choice
        s["tokens"] = near.argmax(-1).to(torch.int32)
        s["logprob"], s["entropy"] = torch.empty(r, device=dev), torch.empty(r, device=dev)
        s["top_ids"] = torch.empty(r, c["top"], dtype=torch.int32, device=dev) if c["top"] else None
        s["top_logprobs"] = torch.empty(r, c["top"], device=dev) if c["top"] else None
        if own:
            s["ws"] = torch.empty(_library().logprobs_workspace_bytes(r, v, c["top"]), dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------ the delta rule, plain form
def _rows(s, size):
    """The token of each place of the sequences padded to `size`, and whether
    there is one."""
    at = torch.arange(size, device="cuda")[None]
    first, end = s["offsets"][:-1, None].long(), s["offsets"][1:, None].long()
    live = first + at < end
    return torch.where(live, first + at, 0), live


def _chunked(s, x, heads):
    """Packed rows [tokens][heads'][..] as [B][heads][chunks][C][..], zero where a
    chunk has no token; value head h reads row h modulo heads'."""
    size = max(1, (max(s["lens"]) + C - 1) // C) * C
    rows, live = _rows(s, size)
    y = x.float()[rows] * live.reshape(live.shape + (1,) * (x.dim() - 1))
    y = y[:, :, torch.arange(heads, device="cuda") % x.shape[1]]
    return y.movedim(2, 1).unflatten(2, (size // C, C))


def _packed(s, y, like):
    """The inverse of _chunked for the tokens there are, into like's shape."""
    rows, live = _rows(s, y.shape[2] * C)
    flat = y.flatten(2, 3).movedim(1, 2)
    out = torch.zeros(like.shape, device="cuda")
    out[rows[live]] = flat[live]
    return out


def _mT(x):
    return x.transpose(-1, -2).contiguous()


def _within(s, c):
    """What a chunk's tokens do to each other: decays, A, P and T = (I + A)^-1."""
    hv = c["hv"]
    w = {n: _chunked(s, s[n], hv) for n in ("q", "k", "v", "beta", "gate")}
    g = w["gate"].double().cumsum(-1)
    w["rise"] = torch.exp(g).float()                       # from the chunk's start to each token
    w["fall"] = torch.exp(g[..., -1:] - g).float()         # from each token to the chunk's end
    low = torch.ones(C, C, dtype=torch.bool, device="cuda").tril()
    w["decay"] = torch.exp((g[..., :, None] - g[..., None, :]).masked_fill(~low, float("-inf"))).float()
    w["kk"] = w["k"] @ _mT(w["k"])
    w["a"] = (w["beta"][..., None] * w["decay"] * w["kk"]).tril(-1)
    w["p"] = SCALE * w["decay"] * (w["q"] @ _mT(w["k"]))
    t = torch.eye(C, device="cuda").expand_as(w["a"]).clone()
    for i in range(1, C):
        t[..., i:i + 1, :] -= w["a"][..., i:i + 1, :i] @ t[..., :i, :].contiguous()
    w["t"] = t
    return w


def _across(s, c, w):
    """The states [B][heads][dk][dv] that enter each chunk and the last one, and
    each token's correction."""
    b, hv, chunks = w["gate"].shape[:3]
    state = torch.zeros(b, hv, D, D, device="cuda") if s["state"] is None else _mT(s["state"])
    states, deltas = [state], []
    for n in range(chunks):
        x = w["v"][:, :, n] - w["rise"][:, :, n, :, None] * (w["k"][:, :, n] @ state)
        delta = w["t"][:, :, n] @ (w["beta"][:, :, n, :, None] * x)
        state = w["rise"][:, :, n, -1, None, None] * state + _mT(w["k"][:, :, n]) @ (w["fall"][:, :, n, :, None] * delta)
        states.append(state)
        deltas.append(delta)
    return torch.stack(states[:-1], 2), torch.stack(deltas, 2), state


def _plain_chunk(s, c):
    w = _within(s, c)
    states, deltas, last = _across(s, c, w)
    y = SCALE * w["rise"][..., None] * (w["q"] @ states) + w["p"] @ deltas
    return {"out": _packed(s, y, s["v"]).to(TYPES[c["type"]]), "state": _mT(last)}


def _plain_backward(s, c):
    w = _within(s, c)
    states, delta, _ = _across(s, c, w)
    do = _chunked(s, s["d_out"], c["hv"])
    ds = torch.zeros_like(states[:, :, 0]) if s["d_state_out"] is None else _mT(s["d_state_out"])
    seed = _mT(w["p"]) @ do
    rise, fall, beta = w["rise"][..., None], w["fall"][..., None], w["beta"][..., None]
    out_q = SCALE * _mT(rise * w["q"]) @ do
    tT, rk = _mT(w["t"]), _mT(rise * w["k"])
    later, rs = [], []
    for n in reversed(range(do.shape[2])):
        later.append(ds)
        r = tT[:, :, n] @ (seed[:, :, n] + fall[:, :, n] * (w["k"][:, :, n] @ ds))
        ds = w["rise"][:, :, n, -1, None, None] * ds + out_q[:, :, n] - rk[:, :, n] @ (beta[:, :, n] * r)
        rs.append(r)
    later, r = torch.stack(later[::-1], 2), torch.stack(rs[::-1], 2)
    sT = _mT(states)
    dp = (do @ _mT(delta)).tril()
    da = -(r @ _mT(delta)).tril(-1)
    pd, e = SCALE * dp * w["decay"], da * beta * w["decay"]
    dq1, dk1, dk2 = SCALE * rise * (do @ sT), -beta * rise * (r @ sT), fall * (delta @ _mT(later))
    dq = dq1 + pd @ w["k"]
    dk = dk1 + dk2 + _mT(pd) @ w["q"] + (e + _mT(e)) @ w["k"]
    pairs = (dp * w["p"] + da * w["a"]).double()
    dbeta = (r * (w["v"] - rise * (w["k"] @ states))).sum(-1) + (da * w["decay"] * w["kk"]).sum(-1)
    end = (dk2 * w["k"]).double().sum(-1)
    dg = (dq1 * w["q"] + dk1 * w["k"]).double().sum(-1) + pairs.sum(-1) - pairs.sum(-2) - end
    dg[..., -1] += end.sum(-1) + w["rise"][..., -1] * (later * states).double().sum((-1, -2))
    dgate = dg.flip(-1).cumsum(-1).flip(-1).float()
    t, hk = TYPES[c["type"]], c["hk"]
    group = lambda x: x.unflatten(1, (c["hv"] // hk, hk)).sum(1)
    out = {"dq": _packed(s, group(dq), s["q"]).to(t), "dk": _packed(s, group(dk), s["k"]).to(t),
           "dv": _packed(s, beta * r, s["v"]).to(t), "dbeta": _packed(s, dbeta, s["beta"]),
           "dgate": _packed(s, dgate, s["gate"])}
    return dict(out, d_state=_mT(ds)) if s["d_state"] is not None else out


def _plain_decode(s, c):
    hv = c["hv"]
    heads = torch.arange(hv, device="cuda") % c["hk"]
    rows, live = _rows(s, c["t"])
    x = {n: s[n].float()[rows] for n in ("q", "k", "v", "beta", "gate")}
    slots = s["slots"].long()
    m, ys = s["state"][slots], []
    for i in range(c["t"]):
        q, k = x["q"][:, i, heads], x["k"][:, i, heads]
        kept = torch.exp(x["gate"][:, i])[..., None, None] * m
        fix = x["beta"][:, i, :, None] * (x["v"][:, i] - (kept * k[:, :, None]).sum(-1))
        m = torch.where(live[:, i, None, None, None], kept + fix[..., None] * k[:, :, None], m)
        ys.append(SCALE * (m * q[:, :, None]).sum(-1))
    y = torch.stack(ys, 1)
    out, state = torch.zeros(s["v"].shape, device="cuda"), s["state"].clone()
    out[rows[live]] = y[live]
    state[slots] = m
    return {"out": out.to(TYPES[c["type"]]), "state": state}


# ------------------------------------------------------- the others, plain form
def _tiles(x, tall):
    """x padded with zeros to whole blocks, as [row blocks][tall][column blocks][BLOCK]."""
    rows, n = x.shape
    y = torch.zeros((rows + tall - 1) // tall * tall, _blocks(n) * BLOCK, dtype=x.dtype, device="cuda")
    y[:rows, :n] = x
    return y.unflatten(1, (-1, BLOCK)).unflatten(0, (-1, tall))


def _plain_quant(s, c):
    x = _tiles(s["x"].double(), c["block_rows"])
    top = x.abs().amax((1, 3), keepdim=True)
    y = torch.where(top > 0, F8_MOST * x / top, 0.0)
    # to three bits behind the first, or to the smallest step
    step = (torch.frexp(y)[1].clamp(min=-5).long() + (1023 - 4) << 52).view(torch.float64)    # a power of two
    scale = (top / F8_MOST).float()
    values = (torch.round(y / step) * step).float() * scale
    return {"values": values.flatten(0, 1).flatten(1, 2)[:c["rows"], :c["n"]].contiguous(), "scale": scale[:, 0, :, 0]}


def _spread(scale, tall, rows, k):
    return scale.repeat_interleave(tall, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :k]


def _plain_linear(s, c):
    a = s["a"].float() * _spread(s["a_scale"], 1, c["m"], c["k"])
    w = s["w"].float() * _spread(s["w_scale"], BLOCK, s["w"].shape[0], c["k"])
    y = a @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return [p.to(TYPES[c["out"]]).contiguous() for p in y.split(_outs(c), 1)]


def _order(x):
    """Whole numbers in the order of the float32 values."""
    b = x.view(torch.int32).long()
    return torch.where(b < 0, -(b & 0x7fffffff), b)


def _plain_logprobs(s, c):
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    z = e.double().sum(-1, keepdim=True)
    base = top.double() + torch.log(z)
    at = lambda ids: (x.gather(1, ids).double() - base).float()
    out = {"logprob": at(s["tokens"].long()[:, None])[:, 0]}
    part = torch.where(e > 0, e * (x - top), 0.0)
    out["entropy"] = (torch.log(z) - part.double().sum(-1, keepdim=True) / z).float()[:, 0]
    if c["top"]:
        ids = torch.arange(c["v"], device="cuda")
        best = torch.topk((_order(x) << 32) - ids, c["top"], dim=1).values
        ids = (-best) & 0xffffffff
        out["top_ids"], out["top_logprobs"] = ids.int(), at(ids)
    return out


def run(state):
    s, c = state, state["case"]
    if c["op"] == "chunk":
        if own:
            _library().chunk(s["q"], s["k"], s["v"], s["beta"], s["gate"], s["out"], state=s["state"],
                             state_out=s["state_out"], offsets=s["offsets"], workspace=s["ws"])
            return {"out": s["out"], "state": s["state_out"]}
        return _plain_chunk(s, c)
    if c["op"] == "backward":
        if own:
            _library().chunk_backward(s["q"], s["k"], s["v"], s["beta"], s["gate"], s["d_out"], s["dq"], s["dk"],
                                      s["dv"], s["dbeta"], s["dgate"], state=s["state"],
                                      d_state_out=s["d_state_out"], d_state=s["d_state"], offsets=s["offsets"],
                                      workspace=s["ws"])
            names = ["dq", "dk", "dv", "dbeta", "dgate"] + (["d_state"] if s["d_state"] is not None else [])
            return {n: s[n] for n in names}
        return _plain_backward(s, c)
    if c["op"] == "decode":
        if own:
            _library().decode(s["q"], s["k"], s["v"], s["beta"], s["gate"], s["out"], s["state"],
                              state_out=s["state_out"], offsets=s["offsets"], slots=s["slots"])
            return {"out": s["out"], "state": s["state_out"]}
        return _plain_decode(s, c)
    if c["op"] == "quant":
        if own:
            _library().quantize_f8(s["x"], s["q"], s["scale"], block_rows=c["block_rows"])
            return {"values": s["q"].float() * _spread(s["scale"], c["block_rows"], c["rows"], c["n"]),
                    "scale": s["scale"]}
        return _plain_quant(s, c)
    if c["op"] == "linear":
        if own:
            _library().linear_f8(s["a"], s["a_scale"], s["w"], s["w_scale"], s["outs"], bias=s["bias"])
            return s["outs"]
        return _plain_linear(s, c)
    if own:
        _library().logprobs(s["logits"], s["tokens"], s["logprob"], s["entropy"], top_ids=s["top_ids"],
                            top_logprobs=s["top_logprobs"], workspace=s["ws"])
        names = ["logprob", "entropy"] + (["top_ids", "top_logprobs"] if c["top"] else [])
        return {n: s[n] for n in names}
    return _plain_logprobs(s, c)


# ------------------------------------------------------------------- in 64 bits
def _exact_rule(s, c):
    """The recurrence token by token on S [B][heads][dk][dv] in 64 bits; the
    gradient by its adjoint, with the states of one segment at a time."""
    hv, longest = c["hv"], max(1, max(s["lens"]))
    heads = torch.arange(hv, device="cuda") % c["hk"]
    rows, live = _rows(s, longest)
    take = lambda name: s[name].double()[rows]
    q, k, v = take("q")[:, :, heads], take("k")[:, :, heads], take("v")
    # a place without a token changes nothing
    beta, e = take("beta") * live[..., None], torch.exp(take("gate") * live[..., None])
    if s["state"] is None:
        now = torch.zeros(c["b"], hv, D, D, dtype=torch.float64, device="cuda")
    else:
        now = (s["state"] if s["slots"] is None else s["state"][s["slots"].long()]).double().transpose(2, 3).contiguous()

    def token(m, t):
        m = e[:, t, :, None, None] * m
        miss = v[:, t] - torch.matmul(k[:, t, :, None], m)[:, :, 0]
        return m + k[:, t, :, :, None] * (beta[:, t, :, None] * miss)[:, :, None], miss

    def packed(x, shape):
        y = torch.zeros(shape, dtype=torch.float64, device="cuda")
        y[rows[live]] = x[live]
        return y

    if c["op"] != "backward":
        y = torch.zeros_like(v)
        for t in range(longest):
            now, _ = token(now, t)
            y[:, t] = torch.matmul(q[:, t, :, None], now)[:, :, 0] / D ** 0.5
        last = now.transpose(2, 3).contiguous()
        if s["slots"] is not None:
            pool = s["state"].double()
            pool[s["slots"].long()] = last
            last = pool
        return {"out": packed(y, s["v"].shape), "state": last}
    seg, marks = 64, []
    for t in range(longest):
        if t % seg == 0:
            marks.append(now)
        now, _ = token(now, t)
    do = take("d_out") * live[..., None, None]
    grad = torch.zeros_like(now) if s["d_state_out"] is None else s["d_state_out"].double().transpose(2, 3).contiguous()
    d = {n: torch.zeros_like(x) for n, x in (("q", q), ("k", k), ("v", v), ("beta", beta), ("gate", e))}
    for first in reversed(range(0, longest, seg)):
        path, now = [], marks[first // seg]
        for t in range(first, min(first + seg, longest)):
            before = now
            now, miss = token(now, t)
            path.append((before, miss, now))
        for t in reversed(range(first, min(first + seg, longest))):
            before, miss, after = path[t - first]
            o = do[:, t] / D ** 0.5
            d["q"][:, t] = torch.matmul(after, o[..., None])[..., 0]
            grad = grad + q[:, t, :, :, None] * o[:, :, None]
            dfix = torch.matmul(k[:, t, :, None], grad)[:, :, 0]
            d["beta"][:, t] = (dfix * miss).sum(-1)
            dmiss = beta[:, t, :, None] * dfix
            d["v"][:, t] = dmiss
            kept = e[:, t, :, None, None] * before
            d["k"][:, t] = (torch.matmul(grad, (beta[:, t, :, None] * miss)[..., None])
                            - torch.matmul(kept, dmiss[..., None]))[..., 0]
            grad = grad - k[:, t, :, :, None] * dmiss[:, :, None]
            d["gate"][:, t] = (grad * kept).sum((-1, -2))
            grad = e[:, t, :, None, None] * grad
    share = lambda x: x.unflatten(2, (hv // c["hk"], c["hk"])).sum(2)
    out = {"dq": packed(share(d["q"]), s["q"].shape), "dk": packed(share(d["k"]), s["k"].shape)}
    for n in ("v", "beta", "gate"):
        out["d" + n] = packed(d[n], s[n].shape)
    if s["d_state"] is not None:
        out["d_state"] = grad.transpose(2, 3).contiguous()
    return out


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    c = case
    s = prepare(case, seed)
    if c["op"] in ("chunk", "backward", "decode"):
        return _exact_rule(s, c)
    if c["op"] == "quant":
        x, tall = s["x"].double(), c["block_rows"]
        whole = torch.nn.functional.pad(x, (0, -c["n"] % BLOCK, 0, -c["rows"] % tall))
        top = whole.reshape(whole.shape[0] // tall, tall, -1, BLOCK).abs().amax(-1).amax(1)
        wide = top.repeat_interleave(tall, 0)[:c["rows"]].repeat_interleave(BLOCK, 1)[:, :c["n"]]
        r = torch.where(wide > 0, x * F8_MOST / wide, torch.zeros_like(x))
        power = torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6)))
        power = torch.where(r.abs() >= torch.exp2(power + 1), power + 1, power)
        unit = torch.exp2(power - 3)
        return {"values": (r / unit).round() * unit * (wide / F8_MOST), "scale": top / F8_MOST}
    if c["op"] == "linear":
        n = s["w"].shape[0]
        y = torch.zeros(c["m"], n, dtype=torch.float64, device="cuda")
        for i in range(_blocks(c["k"])):
            cut = slice(i * BLOCK, min(c["k"], (i + 1) * BLOCK))
            part = torch.matmul(s["a"][:, cut].double(), s["w"][:, cut].double().t().contiguous())
            y += part * s["a_scale"][:, i:i + 1].double() * s["w_scale"][:, i].double().repeat_interleave(BLOCK)[:n]
        if s["bias"] is not None:
            y += s["bias"].double()
        return list(torch.split(y, _outs(c), 1))
    x = s["logits"].double()
    norm = torch.logsumexp(x, -1, keepdim=True)
    lp = x - norm
    out = {"logprob": lp.gather(1, s["tokens"].long()[:, None])[:, 0],
           "entropy": -torch.where(lp > float("-inf"), torch.exp(lp) * lp, torch.zeros_like(lp)).sum(-1)}
    if c["top"]:
        out["top_ids"] = None
        out["top_logprobs"] = torch.sort(lp, dim=1, descending=True).values[:, :c["top"]].contiguous()
    return out


def work(case):
    c = case
    if c["op"] in ("chunk", "backward", "decode"):
        n, z = sum(_lens(c)), SIZES[c["type"]]
        state = 4 * c["b"] * c["hv"] * D * D
        rows = n * D * z * (2 * c["hk"] + 2 * c["hv"]) + 8 * n * c["hv"]
        if c["op"] == "backward":
            # q k v beta gate d_out, and a gradient of each but d_out; a state and its two gradients
            return {"bytes": 2 * rows - n * D * z * c["hv"] + (3 * state if c["start"] else 0),
                    "flops": 18 * n * c["hv"] * D * D}
        # the recurrence's own operations: two products with the state and its update
        return {"bytes": rows + state * (2 if c["op"] == "decode" or c["start"] else 1),
                "flops": 7 * n * c["hv"] * D * D}
    if c["op"] == "quant":
        e = c["rows"] * c["n"]
        return {"bytes": e * (SIZES[c["x"]] + 1) + 4 * e // (BLOCK * c["block_rows"]), "flops": 3 * e}
    if c["op"] == "linear":
        n, k = sum(_outs(c)), c["k"]
        b = (c["m"] + n) * k + 4 * (c["m"] + _blocks(n)) * _blocks(k) + c["m"] * n * SIZES[c["out"]]
        return {"bytes": b + (4 * n if c["bias"] else 0), "flops": 2 * c["m"] * n * k}
    e = c["rows"] * c["v"]
    return {"bytes": e * SIZES[c["logits"]] + c["rows"] * (12 + 8 * c["top"]), "flops": 4 * e}
