"""Calls made while another device than the context's is current (no GPU: the
launches are counted by a stand-in, fake_device.cc)."""

import ctypes

import pytest

import fake_device
from token_sparse_denoising_layer_b200 import abi

N, D, H, F = 8, 256, 2, 128
ADDR = 4096  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    with pytest.MonkeyPatch.context() as m:
        yield fake_device.load(tmp_path_factory.mktemp("fake"), m)


@pytest.fixture
def ctx(lib):
    """A context of device 1; device 0 is current when the test starts."""
    cfg = abi.hsa_model_cfg(N, 16, D, H, F, 1)
    one, out = (ctypes.c_int * 1)(1), ctypes.c_void_p()
    lib.fake_set_device(1)
    assert lib.hsa_create(ctypes.byref(cfg), 1, one, (ctypes.c_int * 1)(N), 1, 0, None, ctypes.byref(out)) == 0
    lib.fake_set_device(0)
    yield out
    lib.hsa_destroy(out)


def _xa():
    return abi.hsa_cross_attn(ADDR, ADDR, ADDR, ADDR, 5)


def _quantised():
    return abi.hsa_layer_weights_quant(*[ADDR] * 8)


def _qk():
    return abi.hsa_qk_rope(1, None, None, 1e-6, ADDR, N, 128, 1)


def _ext(**kw):
    return abi.hsa_block_ext(ADDR, ctypes.pointer(_xa()), kw.get("txt_len"), None, ctypes.pointer(_qk()),
                             ctypes.pointer(_quantised()) if kw.get("quant") else None)


def _block(lib, ctx, ext):
    w = abi.hsa_layer_weights(*[ADDR] * 4)
    return lib.hsa_layer_forward_ext(ctx, ctypes.byref(w), ctypes.byref(ext), ADDR, ADDR, 4, ADDR, ADDR)


def _step(lib, ctx, ext):
    layers = (abi.hsa_layer_weights * 1)(abi.hsa_layer_weights(*[ADDR] * 4))
    caches = (ctypes.c_void_p * 1)(ADDR)
    w = abi.hsa_model_weights(ADDR, ADDR, layers)
    s = abi.hsa_state(*[ADDR] * 9, caches, caches)
    return lib.hsa_step_ext(ctx, ctypes.byref(w), ctypes.byref(s), ctypes.byref(ext), 0, 1.0, 0.0, 1)


def _cross(lib, ctx):
    a = abi.hsa_cross_args(ADDR, None, 4, 1, ADDR, ADDR, D, 0, D, 0, 5, H, None, None, 0.0, ADDR)
    return lib.hsa_cross_attention(ctx, ctypes.byref(a))


@pytest.mark.parametrize("call,launches", [
    (lambda lib, c: lib.hsa_quant_rows(c, ADDR, 0, 4, 64, 64, ADDR, 64, ADDR), 1),
    (lambda lib, c: lib.hsa_linear_quant(c, ADDR, 64, ADDR, 4, 64, ADDR, 64, ADDR, 8, ADDR), 1),
    (lambda lib, c: lib.hsa_ln_gather_quant(c, ADDR, ADDR, 4, ADDR, ADDR, None, None), 1),
    (lambda lib, c: lib.hsa_rope_table(c, ctypes.byref(abi.rope_cfg([64])), None, 4, ADDR), 1),
    (lambda lib, c: lib.hsa_rope(c, ADDR, D, 0, 4, H, ADDR, 4, 64, None, 0, 0, ADDR, D), 1),
    (lambda lib, c: lib.hsa_qk_norm_rope(c, ctypes.byref(_qk()), ADDR, None, 4, None, 0, ADDR, None, 0, ADDR, None, 0,
                                         None), 1),
    (_cross, 1),
    (lambda lib, c: _block(lib, c, _ext()), 12),
    (lambda lib, c: _block(lib, c, _ext(txt_len=ADDR)), 12),
    (lambda lib, c: _block(lib, c, _ext(txt_len=ADDR, quant=True)), 14),
    (lambda lib, c: lib.hsa_layer_forward_ext(c, ctypes.byref(abi.hsa_layer_weights(*[ADDR] * 4)), None, ADDR, ADDR, 4,
                                              ADDR, ADDR), 7),
    (lambda lib, c: _step(lib, c, _ext(txt_len=ADDR, quant=True)), 18),
], ids=["quant_rows", "linear_quant", "ln_gather_quant", "rope_table", "rope", "qk_norm_rope", "cross_attention", "block",
        "block with text length", "8-bit block", "plain block", "step"])
def test_launches_go_to_the_contexts_device(lib, ctx, call, launches):
    before, strays = lib.fake_launches(), lib.fake_strays()
    assert call(lib, ctx) == 0, lib.hsa_last_error(ctx)
    assert lib.fake_launches() - before == launches
    assert lib.fake_strays() == strays
    assert lib.fake_device() == 0  # and the caller's device is current again


def test_a_kernels_attribute_is_set_on_the_device_it_is_noted_for(lib):
    lib.fake_set_device(0)
    assert lib.fake_ensure_smem_limit(1) == 1
    assert lib.fake_ensure_smem_limit(1) == -1  # once per device
    assert lib.fake_ensure_smem_limit(0) == 0
    assert lib.fake_device() == 0
