"""Cross-attention: masks of another width than the keys."""

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
