"""HsaLoop.run and capture with block extensions that differ from iteration to
iteration, as a timestep's modulation does."""

import pytest

from gpu_util import dev, host, need_gpu, torch
from test_gpu_block_ext import _ext_loop
from token_sparse_denoising_layer_b200 import abi, synth

pytestmark = pytest.mark.gpu


def _per_iteration(loop, base):
    """One StepExt an iteration: the base's members with a modulation of its own."""
    out = []
    for i in range(loop.T):
        out.append(abi.StepExt([abi.block_ext(mod=dev(synth.modulation(loop.D, 100 * i + l)), xa=e._keep[1], txt_len=e._keep[2],
                                              qk=e._keep[4], wq=e._keep[5]) for l, e in enumerate(base._keep)]))
    return out


@pytest.mark.parametrize("quant", [False, True])
def test_run_and_capture_take_an_extension_per_iteration(quant):
    need_gpu()
    loop, base, _, x0, g0, _ = _ext_loop(quant)
    exts = _per_iteration(loop, base)
    loop.reset(x0, g0)
    for i in range(loop.T):
        loop.step(i, ext=exts[i])
    want = host(loop.x)
    loop.reset(x0, g0)
    loop.run(ext=exts)
    abi.hsa_sync_check(loop.ctx)
    assert (host(loop.x) == want).all()
    loop.reset(x0, g0)
    loop.run(ext=exts[0])
    assert not (host(loop.x) == want).all()
    loop.capture(ext=exts)
    loop.reset(x0, g0)
    loop.replay()
    torch.cuda.synchronize()
    assert (host(loop.x) == want).all()
    # a part of the loop needs its own iterations only
    loop.reset(x0, g0)
    loop.run(stop=2, ext=exts[:2])
    part = host(loop.x)
    loop.reset(x0, g0)
    for i in range(2):
        loop.step(i, ext=exts[i])
    assert (host(loop.x) == part).all()
    for call in (lambda: loop.run(ext=exts[:-1]), lambda: loop.capture(ext=exts[:-1])):
        before = abi.hsa_kernel_launches(loop.ctx)
        with pytest.raises(ValueError):
            call()
        assert abi.hsa_kernel_launches(loop.ctx) == before
    loop.close()
