"""Tensors that the binding hands over as dense rows: one whose rows are of another
length would be misread, and is refused."""

import pytest

from gpu_util import need_gpu, torch
from token_sparse_denoising_layer_b200 import abi

pytestmark = pytest.mark.gpu


def _ctx(N=6, D=256, H=2):
    return abi.hsa_create(N=N, D=D, H=H, F=64, L=0, T=1, budgets=[1], counts=[N])


def _zeros(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def test_rows_of_another_length_are_refused():
    need_gpu()
    ctx = _ctx()
    bf, i32 = torch.bfloat16, torch.int32
    x, kv = _zeros(6, 256, dtype=bf), _zeros(2, 8, 256, dtype=bf)
    before = abi.hsa_kernel_launches(ctx)
    table = _zeros(6, 64, 2)  # of 128 places
    for call, what in [
            (lambda: abi.hsa_rope_table(ctx, abi.rope_cfg([64]), _zeros(6, 3, dtype=i32), 6, table), "pos"),
            (lambda: abi.hsa_rope_table(ctx, abi.rope_cfg([32, 32]), _zeros(6, 3, dtype=i32), 6, table), "pos"),
            (lambda: abi.hsa_rope(ctx, x, 6, 2, table, 6, 64, x), "table"),
            (lambda: abi.qk_rope(table=table, P=6, rot=64), "table"),
            (lambda: abi.hsa_cross_attention(ctx, _zeros(6, 320, dtype=bf), None, 6, 2, kv, kv, 8, x), "q"),
            (lambda: abi.hsa_qk_norm_rope(ctx, abi.qk_rope(), None, 6, _zeros(6, 320, dtype=bf)), "q"),
            (lambda: abi.hsa_qk_norm_rope(ctx, abi.qk_rope(), None, 6, None, _zeros(6, 512, dtype=bf)), "k_cache")]:
        with pytest.raises(ValueError, match=f"{what} needs rows"):
            call()
    assert abi.hsa_kernel_launches(ctx) == before


def test_other_shapes_of_the_same_rows_are_taken():
    """Flat tensors, rows split into heads or more axes, one row of a wider table, more rows than are used."""
    need_gpu()
    ctx = _ctx()
    bf, i32 = torch.bfloat16, torch.int32
    g = torch.Generator(device="cuda").manual_seed(1)
    pos = torch.randint(0, 99, (6, 3), generator=g, device="cuda", dtype=i32)
    want, got = _zeros(6, 64, 2), _zeros(7, 128)
    abi.hsa_rope_table(ctx, abi.rope_cfg([44, 42, 42]), pos, 6, want)
    abi.hsa_rope_table(ctx, abi.rope_cfg([44, 42, 42]), pos.view(2, 3, 3), 6, got)
    assert torch.equal(got.view(-1)[:768], want.view(-1))
    q = torch.randn(6, 256, generator=g, device="cuda").to(bf)
    a, b = torch.empty_like(q), torch.empty_like(q)
    abi.hsa_rope(ctx, q, 6, 2, want, 6, 128, a)
    abi.hsa_rope(ctx, q, 6, 2, want.view(-1), 6, 128, b)
    assert torch.equal(a, b)
    abi.hsa_rope(ctx, q, 1, 2, want, 1, 64, b)  # the first planes of the one row that is read
    kv = torch.randn(2, 8, 256, generator=g, device="cuda").to(bf)
    abi.hsa_cross_attention(ctx, q, None, 6, 2, kv, kv, 8, a)
    for shape in ((6, 2, 128), (2, 3, 256), (6 * 256,), (1, 6, 256)):
        abi.hsa_cross_attention(ctx, q.view(shape), None, 6, 2, kv, kv, 8, b)
        assert torch.equal(a, b)
    q1, q2, k1, k2 = q.clone(), q.clone().view(6, 2, 128), q.clone(), q.clone().view(1, 6, 256)
    how = abi.qk_rope(table=want, P=6, rot=128)
    abi.hsa_qk_norm_rope(ctx, how, None, 6, q1, k1)
    abi.hsa_qk_norm_rope(ctx, how, None, 6, q2, k2)
    assert torch.equal(q1.view(-1), q2.view(-1)) and torch.equal(k1.view(-1), k2.view(-1))
    abi.hsa_sync_check(ctx)
