"""The operators around the block on the host (no GPU): every call rejects a
NULL context, and the binding rejects wrong types, sizes and host tensors
before anything reaches the library."""

import ctypes
import os
import types

import pytest

torch = pytest.importorskip("torch")

from token_sparse_denoising_layer_b200 import abi  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(abi.LIB_PATH):
        from token_sparse_denoising_layer_b200 import build
        build.build()
    return abi.load()


def test_null_context_is_rejected(lib):
    cfg, how, args = abi.rope_cfg([64]), abi.qk_rope(), abi.hsa_cross_args()
    assert lib.hsa_quant_rows(None, None, 0, 1, 16, 16, None, 16, None) == 1
    assert lib.hsa_linear_quant(None, None, 16, None, 1, 16, None, 16, None, 8, None) == 1
    assert lib.hsa_ln_gather_quant(None, None, None, 1, None, None, None, None) == 1
    assert lib.hsa_rope_table(None, ctypes.byref(cfg), None, 1, None) == 1
    assert lib.hsa_rope(None, None, 128, 0, 1, 1, None, 1, 64, None, 0, 0, None, 128) == 1
    assert lib.hsa_qk_norm_rope(None, ctypes.byref(how), None, None, 1, None, 0, None, None, 0,
                                None, None, 0, None) == 1
    assert lib.hsa_cross_attention(None, ctypes.byref(args)) == 1
    assert "NULL" in lib.hsa_last_error(None).decode()


def _ctx():
    return types.SimpleNamespace(ptr=None, cfg=abi.hsa_model_cfg(8, 16, 128, 1, 64, 0), device=0)


def test_binding_rejects_before_the_library():
    ctx = _ctx()
    b, f = torch.zeros(8, 128, dtype=torch.bfloat16), torch.zeros(8, 128)
    i8, i = torch.zeros(8, 128, dtype=torch.int8), torch.zeros(8, dtype=torch.int32)
    for call, word in [
            (lambda: abi.hsa_quant_rows(ctx, i8, 8, 128, i8, f), "a must be"),
            (lambda: abi.hsa_quant_rows(ctx, b, 8, 128, i8, f), "CUDA"),
            (lambda: abi.hsa_linear_quant(ctx, b, f, 8, 128, i8, f, 8, b), "a must be"),
            (lambda: abi.hsa_rope(ctx, f, 8, 1, f, 8, 128, f), "CUDA"),
            (lambda: abi.hsa_rope(ctx, i8, 8, 1, f, 8, 128, i8), "x must be"),
            (lambda: abi.hsa_rope_table(ctx, abi.rope_cfg([64]), f, 8, f), "pos must be"),
            (lambda: abi.hsa_rope_table(ctx, abi.rope_cfg([64]), i[:7], 8, f), "needs 8"),
            (lambda: abi.hsa_qk_norm_rope(ctx, abi.qk_rope(), None, 8, f), "q must be"),
            (lambda: abi.hsa_qk_norm_rope(ctx, abi.qk_rope(), None, 8, None, i8), "k_cache must be"),
            (lambda: abi.hsa_cross_attention(ctx, b, i, 8, 1, f[None], f[None], 8, b), "k must be"),
            (lambda: abi.rope_cfg([2, 2, 2, 2]), "axes"),
            (lambda: abi.rope_cfg([64], scaling="ntk"), "scaling must be"),
            (lambda: abi.qk_rope(norm="layer"), "norm must be"),
            (lambda: abi.qk_rope(layout="pairs"), "layout must be")]:
        with pytest.raises(ValueError, match=word):
            call()
