"""Frequencies of the rotary table as the kernel gets them, against 50 decimal
digits (no GPU: a stand-in launcher keeps what it was given)."""

import ctypes
import decimal
from decimal import Decimal

import pytest

import fake_device
from token_sparse_denoising_layer_b200 import abi

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    with pytest.MonkeyPatch.context() as m:
        yield fake_device.load(tmp_path_factory.mktemp("fake"), m)


def _exact(dims, base=10000.0, scaling="none", factor=1.0, orig_len=0.0, fast=32.0, slow=1.0):
    """Turns per position of every plane, times 2^64."""
    out = []
    with decimal.localcontext() as c:
        c.prec = 50
        base, factor, orig_len, fast, slow = (Decimal(x) for x in (base, factor, orig_len, fast, slow))
        for dim in dims:
            b = base
            if scaling == "base" and dim > 2:
                b = base * (factor.ln() * dim / (dim - 2)).exp()
            for i in range(dim // 2):
                f = (b.ln() * -2 * i / dim).exp()
                if scaling == "linear":
                    f /= factor
                if scaling == "parts":
                    keep = min(Decimal(1), max(Decimal(0), (orig_len * f / (2 * PI) - slow) / (fast - slow)))
                    f = (1 - keep) * f / factor + keep * f
                out.append(f / (2 * PI) * 2 ** 64)
    return out


@pytest.mark.parametrize("dims,kw", [
    ([128], {}), ([128], dict(base=500000.0)), ([44, 42, 42], {}), ([2], {}), ([2, 2], dict(scaling="base", factor=3.0)),
    ([64], dict(scaling="linear", factor=4.0)), ([64], dict(scaling="base", factor=4.0)), ([96], dict(base=1.0000001)),
    ([128], dict(scaling="parts", factor=8.0, orig_len=8192.0)), ([6, 10], dict(scaling="parts", factor=2.0, orig_len=100.0, fast=4.0)),
    ([128], dict(base=1e300)),
])
def test_frequencies_are_right_to_the_last_bit(lib, dims, kw):
    """Half a unit from the rounding to whole units of 2^-64 turns.  What comes before is a
    few roundings of 64 bits each of a value below 0.16 turns, up to 2^-66.6 turns (0.16 unit) apiece: the power (its exponent's
    rounding grows by |ln f|, but f |ln f| < 0.37), the division by 2 pi, and up to five more of a scaling."""
    cfg = abi.hsa_model_cfg(8, 16, 128, 1, 64, 0)
    one, ctx = (ctypes.c_int * 1)(1), ctypes.c_void_p()
    assert lib.hsa_create(ctypes.byref(cfg), 1, one, (ctypes.c_int * 1)(8), 1, 0, None, ctypes.byref(ctx)) == 0
    pos = None if len(dims) == 1 else 4096
    assert lib.hsa_rope_table(ctx, ctypes.byref(abi.rope_cfg(dims, **kw)), pos, 4, 4096) == 0
    got, want = lib.fake_turns(), _exact(dims, **kw)
    for i, w in enumerate(want):
        assert abs(got[i] - w) <= Decimal(2), (i, got[i], w)
    lib.hsa_destroy(ctx)
