"""Block extensions in the binding, on the host (no GPU): tensors by their
attributes only, as the binding looks at them."""

import types

import pytest

torch = pytest.importorskip("torch")

from token_sparse_denoising_layer_b200 import abi  # noqa: E402

D, N = 128, 8


class OnDevice:
    """What the binding asks a tensor, of one that would lie on CUDA device `where`."""

    def __init__(self, *shape, dtype=torch.float32, where=0):
        self.shape, self.dtype, self.where, self.is_cuda = torch.Size(shape), dtype, where, True

    def get_device(self):
        return self.where

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def view(self, dtype):
        return OnDevice(*self.shape, dtype=dtype, where=self.where)


def _ctx():
    return types.SimpleNamespace(ptr=None, cfg=abi.hsa_model_cfg(N, 16, D, 1, 64, 1), device=0)


def _xa(where=0):
    t = lambda *s: OnDevice(*s, dtype=torch.bfloat16, where=where)  # noqa: E731
    return abi.cross_attn(t(D, D), t(D, D), t(5, D), t(5, D), 5)


def test_a_bool_text_mask_is_taken_as_cross_attention_takes_one():
    for dtype in (torch.bool, torch.uint8):
        s = abi.block_ext(xa=_xa(), txt_mask=OnDevice(5, dtype=dtype))
        assert s.txt_mask == 4096
    with pytest.raises(ValueError, match="txt_mask"):
        abi.block_ext(xa=_xa(), txt_mask=OnDevice(4, dtype=torch.bool))
    with pytest.raises(ValueError, match="txt_mask"):
        abi.block_ext(xa=_xa(), txt_mask=OnDevice(5, dtype=torch.int32))


def test_structs_that_the_caller_filled_are_taken():
    """Their tensors are not known, so only what the library checks is checked."""
    ctx = _ctx()
    abi._check_ext(ctx, abi.hsa_block_ext())
    abi._check_ext(ctx, abi.hsa_block_ext(mod=4096))
    quant = abi.hsa_layer_weights_quant(*[4096] * 8)
    abi._check_ext(ctx, abi.block_ext(qk=abi.hsa_qk_rope(eps=1e-6), wq=quant, xa=abi.hsa_cross_attn(*[4096] * 4, 5)))
    for short in (abi.hsa_qk_rope(table=4096, P=N - 1, rot=16), abi.qk_rope(table=OnDevice(N - 1, 8, 2), P=N - 1, rot=16)):
        with pytest.raises(ValueError, match="row per token"):
            abi._check_ext(ctx, abi.block_ext(qk=short))


@pytest.mark.parametrize("what", ["mod", "txt_len", "txt_mask", "xa", "wq"])
def test_tensors_of_another_device_are_refused(what):
    quant = abi.hsa_layer_weights_quant(*[4096] * 8)

    def ext(where):
        i8 = lambda *s: (OnDevice(*s, dtype=torch.int8, where=where), OnDevice(s[0], where=where))  # noqa: E731
        quant._keep = [i8(3 * D, D), i8(D, D), i8(64, D), i8(D, 64)]
        parts = {"mod": OnDevice(6, D, where=where), "txt_len": OnDevice(1, dtype=torch.int32, where=where),
                 "txt_mask": OnDevice(5, dtype=torch.uint8, where=where), "xa": _xa(where), "wq": quant}
        return abi.block_ext(**{"xa": _xa(), **{what: parts[what]}})

    abi._check_ext(_ctx(), ext(0))
    with pytest.raises(ValueError, match="on cuda:1, the context on cuda:0"):
        abi._check_ext(_ctx(), ext(1))


def test_modulation_and_norm_weights_of_another_shape_are_refused():
    ctx = _ctx()
    for shape in ((6, D), (6 * D,), (1, 6, D), (7, D)):
        abi._check_ext(ctx, abi.block_ext(mod=OnDevice(*shape)))
    for shape in ((6, 2 * D), (5, D), (6, 1, 2 * D)):
        with pytest.raises(ValueError, match="mod needs"):
            abi._check_ext(ctx, abi.block_ext(mod=OnDevice(*shape)))
    two = types.SimpleNamespace(ptr=None, cfg=abi.hsa_model_cfg(N, 16, D, 2, 64, 1), device=0)
    for norm, width in (("head", D // 2), ("row", D)):
        abi._check_qk(two, abi.qk_rope(norm=norm, w_q=OnDevice(width), w_k=OnDevice(1, width)))
        for bad in (width // 2, width + 4, 2 * width):
            with pytest.raises(ValueError, match=f"norm weights need {width}"):
                abi._check_qk(two, abi.qk_rope(norm=norm, w_k=OnDevice(bad)))
    abi._check_qk(two, abi.qk_rope(norm="none", w_q=OnDevice(3)))
