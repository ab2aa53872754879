"""Cross-attention: masks of another width than the keys, and sequences of very
unequal length."""

import pytest

from gpu_util import need_gpu, torch
from token_sparse_denoising_layer_b200 import abi

pytestmark = pytest.mark.gpu


def _ctx(D, H):
    return abi.hsa_create(N=1, D=D, H=H, F=64, L=0, T=1, budgets=[1], counts=[1])


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def test_a_mask_of_another_width_is_refused():
    """States padded further than S are read through their strides; a mask has rows of S bytes."""
    need_gpu()
    B, wide, S, n, D = 3, 96, 80, 12, 128
    ctx = _ctx(D, 1)
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = _randn(g, n, D), _randn(g, B, wide, D), _randn(g, B, wide, D)
    mask = torch.rand(B, wide, generator=g, device="cuda") > 0.4
    o, want = torch.empty_like(q), torch.empty_like(q)
    abi.hsa_cross_attention(ctx, q, None, n, B, k, v, S, want, kv_mask=mask[:, :S].contiguous())
    abi.hsa_cross_attention(ctx, q, None, n, B, k, v, S, o, kv_mask=mask[:, :S].contiguous().view(-1))
    assert torch.equal(o, want)
    for bad in (mask, mask.to(torch.uint8), mask[:, None], torch.cat([mask, mask])[:, :48].contiguous()):
        with pytest.raises(ValueError, match="kv_mask"):
            abi.hsa_cross_attention(ctx, q, None, n, B, k, v, S, o, kv_mask=bad)
    # one sequence's row begins where the mask does, whatever lies behind it
    abi.hsa_cross_attention(ctx, q[:4], None, 4, 1, k, v, S, o, kv_mask=mask[:1])
    assert torch.equal(o[:4], want[:4])
    abi.hsa_sync_check(ctx)


def _sequential64(q, starts, k, v, H, Hk, d):
    o = torch.zeros(q.shape[0], H, d, dtype=torch.float64, device="cuda")
    for b in range(len(starts) - 1):
        rows = slice(starts[b], starts[b + 1])
        for h in range(H):
            c = slice(h // (H // Hk) * d, (h // (H // Hk) + 1) * d)
            p = torch.softmax(q[rows, h * d:(h + 1) * d].double() @ k[b][:, c].double().t() * d ** -0.5, dim=1)
            o[rows, h] = p @ v[b][:, c].double()
    return o.reshape(q.shape[0], H * d)


def _us(f):
    """Least device time of a few calls, in microseconds."""
    best = 1e9
    for _ in range(8):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        b.synchronize()
        best = min(best, 1e3 * a.elapsed_time(b))
    return best


@pytest.mark.parametrize("H,Hk,d,B,n,S", [(2, 2, 128, 64, 64, 1024), (2, 2, 64, 40, 80, 1500), (4, 1, 128, 64, 64, 700),
                                          (2, 2, 128, 64, 256, 1024), (2, 2, 128, 3, 12, 3000)])
@pytest.mark.parametrize("where", [0, 1, -1])
def test_one_long_sequence_among_short_ones(H, Hk, d, B, n, S, where):
    """The rule for few queries looks at their average, and a captured call is replayed
    with other offsets: one sequence that has them all must not make one block walk
    through them alone.  Its rows are then spread over the blocks of the others, each of which
    takes one more pass over the keys; four times the even case's time allows for that twice over."""
    need_gpu()
    D = H * d
    ctx = _ctx(D, H)
    g = torch.Generator(device="cuda").manual_seed(B + n)
    q, k, v = _randn(g, n, D), _randn(g, B, S, Hk * d), _randn(g, B, S, Hk * d)
    o = torch.empty_like(q)
    even = [b * n // B for b in range(B + 1)]
    long = where % B
    skewed = [0] * (long + 1) + [n] * (B - long)
    st = torch.tensor(even, dtype=torch.int32, device="cuda")

    def call():
        abi.hsa_cross_attention(ctx, q, st, n, B, k, v, S, o, kv_heads=Hk)

    t_even = _us(call)
    st.copy_(torch.tensor(skewed))
    t_skewed = _us(call)
    abi.hsa_sync_check(ctx)
    ref = _sequential64(q, skewed, k, v, H, Hk, d)
    # weights and sums in 32 bits, the output rounded once; scores are good to 2^-14 of a weight
    assert bool(((o.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -12).all())
    assert t_skewed <= 4 * t_even + 20, (t_skewed, t_even)


@pytest.mark.parametrize("H,Hk,d,n,starts", [
    (1, 1, 128, 40, [0, 0, 3, 3, 20, 21, 40]), (4, 2, 64, 17, [2, 2, 2, 9, 10, 16, 16, 16, 16, 16]),
    (2, 1, 128, 60, [0, 1, 2, 3, 40, 41, 42, 42, 42, 60] + [60] * 30), (1, 1, 64, 200, list(range(0, 100)) + [180, 200]),
    (3, 1, 128, 5, [0, 5, 5, 5, 5]), (1, 1, 128, 4, [4, 4, 4, 4, 4]), (1, 1, 128, 70, [0] * 35 + [33] + [70] * 36)])
def test_uneven_sequences_of_few_queries(H, Hk, d, n, starts):
    """Every row of every sequence once, rows of none left, with even offsets captured and uneven ones replayed."""
    need_gpu()
    D, B, S = H * d, len(starts) - 1, 150
    ctx = _ctx(D, H) if D % 128 == 0 else abi.hsa_create(N=1, D=128, H=128 // d, F=64, L=0, T=1, budgets=[1], counts=[1])
    H = ctx.cfg.H
    Hk = min(Hk, H)
    D = H * d
    g = torch.Generator(device="cuda").manual_seed(n)
    q, k, v = _randn(g, n, D), _randn(g, B, S, Hk * d), _randn(g, B, S, Hk * d)
    side = torch.cuda.Stream()
    abi.hsa_set_stream(ctx, side)
    st = torch.tensor([min(n, b * max(1, n // B)) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    o = torch.empty_like(q)
    torch.cuda.synchronize()
    abi.hsa_cross_attention(ctx, q, st, n, B, k, v, S, o, kv_heads=Hk)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        abi.hsa_cross_attention(ctx, q, st, n, B, k, v, S, o, kv_heads=Hk)
    st.copy_(torch.tensor(starts))
    o.fill_(6.0)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    abi.hsa_sync_check(ctx)
    ref = _sequential64(q, starts, k, v, H, Hk, d)
    rows = slice(starts[0], starts[-1])
    # P may be rounded to 16 bits where there are many rows a sequence
    assert bool(((o.double() - ref).abs()[rows] <= 2.0 ** -8 * ref.abs()[rows] + 2.0 ** -6).all())
    assert bool((o[:starts[0]] == 6.0).all()) and bool((o[starts[-1]:] == 6.0).all())
    del graph
