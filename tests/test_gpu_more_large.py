"""GPU: the packed operators on tensors past 2^31 elements.  What lies at the end of
a large call has the bits that a small call gives, whose values other tests check."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_deltanet_decode_amd as g
    return g


@pytest.fixture(autouse=True)
def freed():
    yield
    torch.cuda.empty_cache()


def e(*s, t=torch.float32):
    return torch.empty(*s, dtype=t, device="cuda")


def tokens(n):
    """bf16 tokens of 32 and 16 heads, and beta and gate."""
    q, k = (torch.nn.functional.normalize(e(n, 16, 128, t=BF16).normal_(), dim=-1) for _ in range(2))
    return [q, k, e(n, 32, 128, t=BF16).normal_(), e(n, 32).uniform_(), e(n, 32).uniform_(-1, 0)]


def test_chunk(g):
    torch.manual_seed(0)
    n, last = 560_000, 200                                # v and out: 2.3e9 elements
    x, state = tokens(n), e(2, 32, 128, 128).normal_()
    out, so = e(n, 32, 128, t=BF16), torch.empty_like(state)
    offsets = torch.tensor([0, n - last, n], dtype=torch.int32, device="cuda")
    g.chunk(*x, out, state=state, state_out=so, offsets=offsets, workspace=e(g.chunk_workspace_bytes(2, n, BF16), t=torch.uint8))
    y, s = e(1, last, 32, 128, t=BF16), e(1, 32, 128, 128)
    g.chunk(*(t[None, n - last:].contiguous() for t in x), y, state=state[1:], state_out=s,
            workspace=e(g.chunk_workspace_bytes(1, last, BF16), t=torch.uint8))
    assert torch.equal(out[n - last:], y[0]) and torch.equal(so[1:], s)


def test_chunk_backward(g):
    torch.manual_seed(1)
    n, last = 530_000, 200                                # states: 4.3e9 floats
    x, d_out = tokens(n), e(n, 32, 128, t=BF16).normal_()
    grads = [torch.empty_like(t) for t in x]
    ds = e(2, 32, 128, 128)
    offsets = torch.tensor([0, n - last, n], dtype=torch.int32, device="cuda")
    need = g.chunk_backward_workspace_bytes(2, n, BF16)
    g.chunk_backward(*x, d_out, *grads, d_state=ds, offsets=offsets, workspace=e(need, t=torch.uint8))
    small = [t[None, n - last:].contiguous() for t in x]
    want, s = [torch.empty_like(t) for t in small], e(1, 32, 128, 128)
    g.chunk_backward(*small, d_out[None, n - last:].contiguous(), *want, d_state=s,
                     workspace=e(g.chunk_backward_workspace_bytes(1, last, BF16), t=torch.uint8))
    assert all(torch.equal(a[n - last:], b[0]) for a, b in zip(grads, want)) and torch.equal(ds[1:], s)


def test_decode(g):
    torch.manual_seed(2)
    pool = e(4200, 32, 128, 128)                          # 2.2e9 floats
    x = [t[:, None].contiguous() for t in tokens(3)]
    slots = torch.tensor([4199, 7, 4100], dtype=torch.int32, device="cuda")
    state = e(3, 32, 128, 128).normal_()
    pool[slots.long()] = state
    out, y = e(3, 1, 32, 128, t=BF16), e(3, 1, 32, 128, t=BF16)
    g.decode(*x, out, pool, slots=slots)
    g.decode(*x, y, state)
    assert torch.equal(out, y) and torch.equal(pool[slots.long()], state)


def test_codes_and_product(g):
    torch.manual_seed(3)
    M, K, N = 180_000, 256, 12_352                        # outputs: 2.2e9 elements
    x, w = e(M, K, t=BF16).normal_(), e(N, K).normal_()
    q, s, wq, ws = e(M, K, t=F8), e(M, 2), e(N, K, t=F8), e(97, 2)
    g.quantize_f8(x, q, s)
    g.quantize_f8(w, wq, ws, block_rows=128)
    out, last = e(M, N, t=BF16), e(5_000, N, t=BF16)
    g.linear_f8(q, s, wq, ws, out)
    g.linear_f8(q[-5000:], s[-5000:], wq, ws, last)       # (tiles of the same size)
    assert torch.equal(out[-5000:], last)
    del w, last
    q, s = e(M, N, t=F8), e(M, 97)
    g.quantize_f8(out, q, s)
    tail, ts = e(100, N, t=F8), e(100, 97)
    g.quantize_f8(out[-100:], tail, ts)
    assert torch.equal(q[-100:].view(torch.uint8), tail.view(torch.uint8)) and torch.equal(s[-100:], ts)


def test_logprobs(g):
    torch.manual_seed(4)
    rows, V, last = 17_000, 131_071, 2_000                # 2.2e9 logits, one unit a row in both calls
    x = e(rows, V, t=BF16).normal_(std=3)

    def call(x):
        n = x.shape[0]
        r = [e(n), e(n), e(n, 20, t=torch.int32), e(n, 20)]
        g.logprobs(x, torch.full((n,), V - 1, dtype=torch.int32, device="cuda"), *r)
        return r
    assert all(torch.equal(a[-last:], b) for a, b in zip(call(x), call(x[-last:])))
