"""A row that hsa_qk_norm_rope skips is skipped whole: its query, key and value
are judged together, so the cache never keeps a new value beside an old key."""

import pytest

from gpu_util import need_gpu, torch
from token_sparse_denoising_layer_b200 import abi

pytestmark = pytest.mark.gpu

N, D, P = 6, 128, 5


def _call(idx, pos=None, in_place=False, norm="head", table=True, want=7):
    """Queries, both caches and the sources after one call with caches of 3 and queries of 9."""
    ctx = abi.hsa_create(N=N, D=D, H=1, F=64, L=0, T=1, budgets=[1], counts=[N])
    g = torch.Generator(device="cuda").manual_seed(4)
    n = len(idx)
    qkv = torch.randn(n, 3 * D, generator=g, device="cuda").to(torch.bfloat16)
    a = torch.rand(P, D // 2, generator=g, device="cuda") * 6.28
    t = torch.stack([torch.cos(a), torch.sin(a)], dim=-1).contiguous() if table else None
    kc, vc = (torch.full((N, D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.full((n, D), 9.0, dtype=torch.bfloat16, device="cuda")
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    how = abi.qk_rope(norm=norm, table=t, P=P if table else 0, rot=D if table else 0)
    abi.hsa_qk_norm_rope(ctx, how, i32(idx), n, q, kc, vc, q_in=qkv[:, :D], k_in=None if in_place else qkv[:, D:2 * D],
                         v_in=qkv[:, 2 * D:], pos=i32(pos))
    if want:
        with pytest.raises(abi.HsaError) as e:
            abi.hsa_sync_check(ctx)
        assert e.value.status == want
    abi.hsa_sync_check(ctx)
    return q, kc, vc, qkv[:, 2 * D:]


def _check(idx, good, q, kc, vc, v_in):
    old = torch.full((D,), 3.0, dtype=torch.bfloat16, device="cuda")
    written = {r: m for m, r in enumerate(idx) if good[m]}
    for m, ok in enumerate(good):
        assert bool((q[m] == 0).all()) != ok, m
    for r in range(N):
        if r in written:
            assert torch.equal(vc[r], v_in[written[r]]) and not torch.equal(kc[r], old), r
        else:
            assert torch.equal(vc[r], old) and torch.equal(kc[r], old), r


@pytest.mark.parametrize("idx,pos,good", [
    ([0, -1, 6, 2], None, [True, False, False, True]),             # cache rows
    ([0, 1, 2, 5], None, [True, True, True, False]),               # cache row 5 is there, table row 5 is not
    ([3, 1, 0, 5], [4, 5, -1, 0], [True, False, False, True]),     # table rows given
])
@pytest.mark.parametrize("norm", ["head", "row", "none"])
def test_a_bad_row_is_skipped_whole(idx, pos, good, norm):
    need_gpu()
    _check(idx, good, *_call(idx, pos, norm=norm))


@pytest.mark.parametrize("table", [True, False])
def test_a_row_out_of_order_is_skipped_whole_in_place(table):
    need_gpu()
    idx = [0, 2, 2, 1]
    _check(idx, [True, True, False, False], *_call(idx, in_place=True, table=table, norm="head"))


def test_order_does_not_matter_with_keys_from_elsewhere():
    need_gpu()
    idx = [4, 2, 3, 1]
    _check(idx, [True] * 4, *_call(idx, want=0))


def test_without_a_table_its_rows_do_not_matter():
    need_gpu()
    idx = [0, 5, 1, 2]
    _check(idx, [True] * 4, *_call(idx, pos=[0, 99, -3, 2], table=False, want=0))
