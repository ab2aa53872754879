"""The rotary table at the ends of the int32 range."""

from decimal import Decimal, localcontext
import math

import numpy as np
import pytest

from gpu_util import need_gpu, torch
from token_sparse_denoising_layer_b200 import abi

pytestmark = pytest.mark.gpu

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.mark.parametrize("sign", [1, -1])
def test_far_positions_have_no_angle_error_of_their_own(sign):
    """The mean error of a plane's angle over 4096 positions near 2^31.  A frequency is right to a unit of
    2^-64 turns, so its part is 2^-33 turns (7e-10 rad), and the cut of the product to 32 bits adds as much again on average; the
    fp32 roundings of an entry stay below 2^-22 and average out, to five deviations of
    1.2e-7 / 64 at most: 2^-26 in all.  (An error of 2^-56 turns a position, a double's, makes 1e-7.)"""
    need_gpu()
    ctx = abi.hsa_create(N=1, D=128, H=1, F=64, L=0, T=1, budgets=[1], counts=[1])
    n, dim = 4096, 128
    rng = np.random.default_rng(7)
    pos = sign * (2 ** 31 - 1 - rng.integers(0, 2 ** 24, n))
    table = torch.empty(n, dim // 2, 2, device="cuda")
    abi.hsa_rope_table(ctx, abi.rope_cfg([dim]), torch.tensor(pos, dtype=torch.int32, device="cuda")[:, None], n, table)
    abi.hsa_sync_check(ctx)
    got = table.double().cpu().numpy()
    with localcontext() as c:
        c.prec = 60
        turns = [int((Decimal(10000).ln() * -2 * i / dim).exp() / (2 * PI) * 2 ** 120) for i in range(dim // 2)]
    worst = 0.0
    for i, t in enumerate(turns):
        # the angle's fraction of a turn, from whole numbers
        ang = 2 * math.pi * np.array([((int(p) * t) % 2 ** 120 >> 60) / 2.0 ** 60 for p in pos])
        worst = max(worst, float(np.abs(got[:, i, 0] - np.cos(ang)).max()), float(np.abs(got[:, i, 1] - np.sin(ang)).max()))
        mean = float(np.mean(np.cos(ang) * got[:, i, 1] - np.sin(ang) * got[:, i, 0]))
        assert abs(mean) <= 2.0 ** -26, (i, mean)
    assert worst <= 2.0 ** -22
