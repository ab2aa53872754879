"""GPU tests of the operators around the block: 8-bit products with scales,
rotary positions, query/key norm with rotation and cache write, and ragged
cross-attention, each against a plain implementation in 64 bits.

Tolerances are counted in roundings.  One rounding to a type is off by at most
half a step, eps / 2 relative: 2^-8 for bf16, 2^-24 for fp32.
"""

import math

import numpy as np
import pytest

from gpu_util import dev, need_gpu, torch
from token_sparse_denoising_layer_b200 import abi

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8   # one rounding to bf16
F32 = 2.0 ** -24  # one rounding to fp32


def _ctx(N=1, D=128, H=1, **kw):
    return abi.hsa_create(N=N, D=D, H=H, F=64, L=0, T=1, budgets=[1], counts=[N], **kw)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _within(got, want, tol):
    """Every element of got within tol (tensor or number) of want, in 64 bits."""
    bad = (got.double() - want.double()).abs() > tol
    assert not bool(torch.isnan(got.double()).any())
    assert not bool(bad.any()), (int(bad.sum()), float((got.double() - want).abs().max()))


# ---------------------------------------------------------------- 8-bit rows

def _quantised(a):
    """The definition in fp32, on the host: numpy's divisions and products are IEEE."""
    a = a.float().cpu().numpy()
    with np.errstate(all="ignore"):
        top = np.abs(a).max(1).astype(np.float32)
        bad = ~np.isfinite(a).all(1)
        tiny = top < np.float32(2.0 ** -100)
        mul = np.where(tiny | bad, np.float32(0), np.float32(127) / np.where(tiny | bad, 1, top).astype(np.float32))
        q = np.rint((np.where(np.isfinite(a), a, 0) * mul[:, None]).astype(np.float32)).astype(np.int8)
        scale = np.where(tiny, np.float32(0), top / np.float32(127)).astype(np.float32)
    q[bad] = 0
    scale[bad] = np.nan
    return q, scale


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,K", [(1, 1), (3, 7), (9, 8), (130, 129), (33, 1536), (5, 2304), (7, 2312), (6, 8960),
                                 (3, 9217), (2, 40008), (1, 131071), (19, 503), (18, 505), (9, 1015), (9, 1017), (9, 2041),
                                 (5, 3039), (5, 3041), (6, 4063), (6, 4065), (5, 5087), (5, 5089), (5, 8161), (4, 32639), (4, 32641), (40, 3), (20, 62), (9999, 65), (9475, 248), (9473, 249), (9474, 503)])
def test_quant_rows(n, K, dtype):
    need_gpu()
    ctx = _ctx()
    g = _gen(n * 7 + K)
    ld = (K + 15) // 16 * 16 + 16
    a = _randn(g, n, K, dtype=dtype)
    q = torch.full((n, ld), 99, dtype=torch.int8, device="cuda")
    s = torch.empty(n, device="cuda")
    want_q, want_s = _quantised(a)
    padded = torch.full((n, ld), float("nan"), dtype=dtype, device="cuda")  # aligned rows, poison behind them
    padded[:, :K] = a
    for src in (a, padded):
        q.fill_(99)
        abi.hsa_quant_rows(ctx, src, n, K, q, s)
        abi.hsa_sync_check(ctx)
        assert (q[:, :K].cpu().numpy() == want_q).all()
        assert (s.cpu().numpy() == want_s).all()
        assert bool((q[:, K:] == 99).all())  # bytes behind the row are left as they were


def test_quant_rows_extremes():
    need_gpu()
    ctx = _ctx()
    K = 40
    a = torch.zeros(8, K, device="cuda")
    a[1, 3] = float("inf")
    a[2, 5] = float("nan")
    a[2, 6] = float("-inf")
    a[3, 0] = 2.0 ** -101
    a[4, 0] = 2.0 ** -100
    a[4, 1] = -2.0 ** -100
    a[5] = torch.linspace(-3.4e38, 3.4e38, K)
    a[6, 0], a[6, 1], a[6, 2] = 127.0, 0.5, 1.5   # halves go to even: 0 and 2
    a[7] = -1e-30
    want_q, want_s = _quantised(a)
    q, s = torch.empty(8, 48, dtype=torch.int8, device="cuda"), torch.empty(8, device="cuda")
    abi.hsa_quant_rows(ctx, a, 8, K, q, s)
    got_s = s.cpu().numpy()
    assert (q[:, :K].cpu().numpy() == want_q).all()
    assert ((got_s == want_s) | (np.isnan(got_s) & np.isnan(want_s))).all()
    assert np.isnan(got_s[1]) and np.isnan(got_s[2]) and got_s[0] == 0 and got_s[3] == 0
    assert list(q[6, :3].cpu()) == [127, 0, 2] and abs(int(q[4, 0])) == 127


@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (1, 1536, 8960), (2, 40, 33), (5, 17, 8), (8, 8960, 100), (9, 128, 256),
                                   (64, 300, 70), (127, 129, 31), (129, 128, 128), (130, 513, 1000), (256, 256, 256),
                                   (700, 1536, 4608), (1000, 2000, 520), (3000, 64, 2047), (20000, 1536, 1536),
                                   (16, 131071, 24)])
def test_linear_quant(M, K, N):
    """The integer sum is exact; three fp32 roundings and one to bf16 follow."""
    need_gpu()
    ctx = _ctx()
    g = _gen(M + K + N)
    ld = (K + 15) // 16 * 16
    a = torch.randint(-127, 128, (M, ld), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (N, ld + 16), generator=g, device="cuda", dtype=torch.int8)  # bytes past K are junk
    sa = torch.rand(M, generator=g, device="cuda") + 0.1
    sw = torch.rand(N, generator=g, device="cuda") + 0.1
    out = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    abi.hsa_linear_quant(ctx, a, sa, M, K, w, sw, N, out)
    abi.hsa_sync_check(ctx)
    ref = a[:, :K].double() @ w[:, :K].double().t() * sa.double()[:, None] * sw.double()
    _within(out[:M * N].view(M, N), ref, (BF + 4 * F32) * ref.abs())
    assert bool((out[M * N:] == 7.0).all())
    again = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    abi.hsa_linear_quant(ctx, a, sa, M, K, w, sw, N, again)
    assert torch.equal(again, out[:M * N].view(M, N))


def test_linear_quant_largest_sums():
    """The largest sums that 131071 products of bytes can reach stay in 32 bits."""
    need_gpu()
    ctx = _ctx()
    K = 131071
    for M in (2, 200):
        a = torch.full((M, K + 1), -128, dtype=torch.int8, device="cuda")
        w = torch.full((32, K + 1), -128, dtype=torch.int8, device="cuda")
        one = torch.ones(M, device="cuda")
        out = torch.empty(M, 32, dtype=torch.bfloat16, device="cuda")
        abi.hsa_linear_quant(ctx, a, one, M, K, w, one[:1].repeat(32), 32, out)
        _within(out, torch.full_like(out, 1.0).double() * (K * 16384.0), (BF + 4 * F32) * K * 16384.0)


def test_linear_quant_of_a_bad_row_is_nan_in_that_row_alone():
    need_gpu()
    ctx = _ctx()
    g = _gen(5)
    a = _randn(g, 40, 64, dtype=torch.bfloat16)
    a[7, 3] = float("inf")
    w = torch.randint(-127, 128, (48, 64), generator=g, device="cuda", dtype=torch.int8)
    q, s = torch.empty(40, 64, dtype=torch.int8, device="cuda"), torch.empty(40, device="cuda")
    out = torch.empty(40, 48, dtype=torch.bfloat16, device="cuda")
    abi.hsa_quant_rows(ctx, a, 40, 64, q, s)
    abi.hsa_linear_quant(ctx, q, s, 40, 64, w, torch.ones(48, device="cuda"), 48, out)
    nan = torch.isnan(out.float())
    assert bool(nan[7].all()) and int(nan.sum()) == 48


@pytest.mark.parametrize("N,D,a", [(700, 256, 333), (300, 128, 1), (100, 1536, 77), (40, 2048, 40), (30, 5120, 30), (20, 640, 9)])
@pytest.mark.parametrize("mod", [False, True])
def test_ln_gather_quant(N, D, a, mod):
    """The dequantised row is within half a step of the row's scale of LN in 64
    bits, plus fp32 error of the statistics (D terms: far below 2^-14 of the top)."""
    need_gpu()
    ctx = _ctx(N, D, D // 128)
    g = _gen(N + D)
    x = 3 * _randn(g, N, D) + 0.5
    idx = torch.sort(torch.randperm(N, generator=g, device="cuda")[:a]).values.to(torch.int32)
    sh, sc = (0.3 * _randn(g, D), 0.3 * _randn(g, D)) if mod else (None, None)
    q, s = torch.empty(a, D, dtype=torch.int8, device="cuda"), torch.empty(a, device="cuda")
    abi.hsa_ln_gather_quant(ctx, x, idx, a, q, s, sh, sc)
    abi.hsa_sync_check(ctx)
    u = x[idx.long()].double()
    u = (u - u.mean(1, keepdim=True)) / torch.sqrt(u.var(1, unbiased=False, keepdim=True) + 1e-5)
    if mod:
        u = u * (1 + sc.double()) + sh.double()
    top = u.abs().amax(1, keepdim=True)
    assert bool((q.abs().amax(1) == 127).all())
    _within(q.double() * s.double()[:, None], u, top * (0.5 / 127 + 2.0 ** -14))


# ---------------------------------------------------------------- rotary positions

def _freqs(dims, base=10000.0, scaling="none", factor=1.0, orig_len=0.0, fast=32.0, slow=1.0):
    """Frequencies of every plane and their axis, in 64 bits."""
    out = []
    for x, dim in enumerate(dims):
        b = base * factor ** (dim / (dim - 2)) if scaling == "base" and dim > 2 else base
        for i in range(dim // 2):
            f = b ** (-2.0 * i / dim)
            if scaling == "linear":
                f /= factor
            if scaling == "parts":
                r = orig_len * f / (2 * math.pi)
                keep = min(1.0, max(0.0, (r - slow) / (fast - slow)))
                f = (1 - keep) * f / factor + keep * f
            out.append((f, x))
    return out


@pytest.mark.parametrize("dims,kw", [
    ([128], {}), ([16], dict(base=500000.0)), ([44, 42, 42], {}), ([2, 2], dict(scaling="base", factor=3.0)),
    ([64], dict(scaling="linear", factor=4.0)), ([64], dict(scaling="base", factor=4.0)),
    ([128], dict(scaling="parts", factor=8.0, orig_len=8192.0, amp=1.2)),
    ([6, 10], dict(scaling="parts", factor=2.0, orig_len=100.0, fast=4.0)),
])
@pytest.mark.parametrize("P", [1, 300, 5000])
def test_rope_table(dims, kw, P):
    """Reduced angles: sine and cosine of half turns are good to 2 units in the
    last place of a value up to 1 (2^-23 each), then two more roundings."""
    need_gpu()
    ctx = _ctx()
    amp = kw.get("amp", 1.0)
    pos = torch.randint(-1000, 1 << 20, (P, len(dims)), generator=_gen(P), device="cuda", dtype=torch.int32)
    pos[0] = 0
    table = torch.empty(P, sum(dims) // 2, 2, device="cuda")
    abi.hsa_rope_table(ctx, abi.rope_cfg(dims, **kw), pos, P, table)
    abi.hsa_sync_check(ctx)
    fr = _freqs(dims, **{k: v for k, v in kw.items() if k != "amp"})
    ang = torch.stack([pos[:, x].double() * f for f, x in fr], dim=1)
    ref = amp * torch.stack([torch.cos(ang), torch.sin(ang)], dim=-1)
    _within(table, ref, amp * 2.0 ** -21)
    assert bool((table[0, :, 1] == 0).all()) and bool((table[0, :, 0] == np.float32(amp)).all())
    if len(dims) == 1:  # positions 0 .. P-1 when none are given
        t2, t3 = torch.empty_like(table), torch.empty_like(table)
        abi.hsa_rope_table(ctx, abi.rope_cfg(dims, **kw), None, P, t2)
        abi.hsa_rope_table(ctx, abi.rope_cfg(dims, **kw), torch.arange(P, dtype=torch.int32, device="cuda")[:, None], P, t3)
        assert torch.equal(t2, t3)


def _table(g, P, rot):
    a = torch.rand(P, rot // 2, generator=g, device="cuda") * 6.28
    return torch.stack([torch.cos(a), torch.sin(a)], dim=-1).contiguous()


def _turned(x, t, layout):
    """x [n, H, d], t [n, rot/2, 2] in 64 bits; also sum of the magnitudes of each output's two terms."""
    half = t.shape[1]
    c, s = t[:, None, :, 0], t[:, None, :, 1]
    y, mag = x.clone(), x.abs()
    i = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    u, v = x[..., i[0]], x[..., i[1]]
    y[..., i[0]], y[..., i[1]] = u * c - v * s, v * c + u * s
    mag[..., i[0]], mag[..., i[1]] = (u * c).abs() + (v * s).abs(), (v * c).abs() + (u * s).abs()
    return y, mag


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,H,heads,d,rot", [(1, 1, 1, 128, 128), (7, 2, 3, 64, 32), (300, 12, 12, 128, 128),
                                             (65, 2, 2, 64, 64), (33, 4, 5, 128, 48), (10, 2, 40, 64, 16)])
def test_rope(n, H, heads, d, rot, layout, dtype):
    need_gpu()
    ctx = _ctx(1, H * d, H) if (H * d) % 128 == 0 else _ctx(1, 128, 128 // d)
    g = _gen(n + heads)
    wide = _randn(g, n, heads * d + 24, dtype=dtype)
    x = wide[:, 8:8 + heads * d]  # strided rows
    P = n + 9
    table = _table(g, P, rot)
    pos = torch.randint(0, P, (n,), generator=g, device="cuda", dtype=torch.int32)
    eps = BF if dtype == torch.bfloat16 else 0.0
    for p in (None, pos):
        t = table[:n] if p is None else table[p.long()]
        ref, mag = _turned(x.double().reshape(n, heads, d), t.double(), layout)
        out = torch.empty(n, heads * d, dtype=dtype, device="cuda")
        abi.hsa_rope(ctx, x, n, heads, table, P, rot, out, layout=layout, pos=p)
        abi.hsa_sync_check(ctx)
        _within(out.view(n, heads, d), ref, eps * ref.abs() + 4 * F32 * mag)
        assert torch.equal(out.view(n, heads, d)[..., rot:], x.reshape(n, heads, d)[..., rot:])
        # the inverse is the transpose: <R x, y> = <x, R' y>, and R' R x = x
        back = torch.empty_like(out)
        abi.hsa_rope(ctx, out, n, heads, table, P, rot, back, layout=layout, pos=p, inverse=True)
        t2 = t.double().clone()
        t2[..., 1] *= -1
        ref2, mag2 = _turned(out.double().view(n, heads, d), t2, layout)
        _within(back.view(n, heads, d), ref2, eps * ref2.abs() + 4 * F32 * mag2)
        abi.hsa_rope(ctx, out, n, heads, table, P, rot, out, layout=layout, pos=p, inverse=True)  # in place
        assert torch.equal(out, back)


def test_rope_gradient_is_the_inverse():
    """d/dx <w, R x> by central differences of the forward call against the inverse call (fp32, step 1/2: R is linear)."""
    need_gpu()
    ctx = _ctx()
    g = _gen(3)
    x, w, table = _randn(g, 1, 128), _randn(g, 1, 128), _table(g, 1, 64)
    grad = torch.empty_like(w)
    abi.hsa_rope(ctx, w, 1, 1, table, 1, 64, grad, layout="interleaved", inverse=True)
    rows = torch.cat([x + 0.5 * torch.eye(128, device="cuda"), x - 0.5 * torch.eye(128, device="cuda")]).contiguous()
    out = torch.empty_like(rows)
    abi.hsa_rope(ctx, rows, 256, 1, table, 1, 64, out, layout="interleaved",
                 pos=torch.zeros(256, dtype=torch.int32, device="cuda"))
    diff = ((out[:128].double() - out[128:].double()) * w.double()).sum(1)
    # each output carries 3 roundings of values below 8
    _within(grad[0], diff, 2 * 3 * F32 * 8 * float(w.abs().sum()))


def test_rope_reports_table_rows_out_of_range():
    need_gpu()
    ctx = _ctx()
    g = _gen(1)
    x, table = _randn(g, 4, 128, dtype=torch.bfloat16), _table(g, 4, 128)
    out = torch.full_like(x, 5.0)
    abi.hsa_rope(ctx, x, 4, 1, table, 4, 128, out, pos=torch.tensor([0, 4, -1, 3], dtype=torch.int32, device="cuda"))
    with pytest.raises(abi.HsaError) as e:
        abi.hsa_sync_check(ctx)
    assert e.value.status == 7
    assert bool((out[1:3] == 5.0).all()) and not bool((out[0] == 5.0).any())
    abi.hsa_sync_check(ctx)


# ---------------------------------------------------------------- norm, rotation, cache write

def _norm64(x, w, norm, eps, H, d):
    x = x.double()
    if norm == "row":
        x = x / torch.sqrt((x * x).mean(1, keepdim=True) + eps) * (1.0 if w is None else w.double())
    x = x.reshape(-1, H, d)
    if norm == "head":
        x = x / torch.sqrt((x * x).mean(2, keepdim=True) + eps) * (1.0 if w is None else w.double())
    return x


def _qk_ref(x, w, norm, eps, H, d, t, layout):
    """Value and tolerance: one rounding to bf16; the norm's fp32 sum of up to
    10240 squares over 32 lanes and its root are good to 2^-14 at worst."""
    y = _norm64(x, w, norm, eps, H, d)
    y, mag = (y, y.abs()) if t is None else _turned(y, t.double(), layout)
    return y.reshape(len(x), -1), (BF * y.abs() + 2.0 ** -14 * mag).reshape(len(x), -1)


@pytest.mark.parametrize("norm,layout,rot", [("head", "half", 1.0), ("row", "interleaved", 1.0), ("none", "half", 0.25),
                                             ("head", "interleaved", 0.5), ("row", "half", 0.0)])
@pytest.mark.parametrize("N,n,H,d", [(256, 128, 2, 64), (50, 1, 1, 128), (300, 299, 12, 128), (64, 64, 24, 64),
                                     (40, 13, 40, 128), (20, 7, 80, 128), (33, 20, 6, 128), (9, 9, 34, 64)])
def test_qk_norm_rope(N, n, H, d, norm, layout, rot):
    need_gpu()
    D, rot = H * d, int(rot * d)
    ctx = _ctx(N, D, H)
    g = _gen(N + H)
    qkv = _randn(g, n, 3 * D, dtype=torch.bfloat16)
    idx = torch.sort(torch.randperm(N, generator=g, device="cuda")[:n]).values.to(torch.int32)
    width = D if norm == "row" else d
    wq, wk = 1 + 0.1 * _randn(g, width), 1 + 0.1 * _randn(g, width)
    table = _table(g, N + 3, rot) if rot else None
    kc, vc = _randn(g, N, D, dtype=torch.bfloat16), _randn(g, N, D, dtype=torch.bfloat16)
    kc0, vc0 = kc.clone(), vc.clone()
    how = abi.qk_rope(norm=norm, w_q=wq, w_k=wk, eps=1e-5, table=table, P=N + 3 if rot else 0, rot=rot, layout=layout)
    q = torch.empty(n, D, dtype=torch.bfloat16, device="cuda")
    abi.hsa_qk_norm_rope(ctx, how, idx, n, q, kc, vc, q_in=qkv[:, :D], k_in=qkv[:, D:2 * D], v_in=qkv[:, 2 * D:])
    abi.hsa_sync_check(ctx)
    rows = idx.long()
    t = table[rows] if rot else None
    ref_q, tol_q = _qk_ref(qkv[:, :D], wq, norm, 1e-5, H, d, t, layout)
    ref_k, tol_k = _qk_ref(qkv[:, D:2 * D], wk, norm, 1e-5, H, d, t, layout)
    _within(q, ref_q, tol_q)
    _within(kc[rows], ref_k, tol_k)
    assert torch.equal(vc[rows], qkv[:, 2 * D:])
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert torch.equal(kc[rest], kc0[rest]) and torch.equal(vc[rest], vc0[rest])
    # in place: the raw rows written first, then turned where they lie, bit for bit the same
    q2, kc2 = qkv[:, :D].contiguous(), kc0.clone()
    kc2[rows] = qkv[:, D:2 * D]
    abi.hsa_qk_norm_rope(ctx, how, idx, n, q2, kc2)
    abi.hsa_sync_check(ctx)
    assert torch.equal(q2, q) and torch.equal(kc2, kc)
    # explicit table rows, keys alone, no index list
    if rot:
        pos = torch.randint(0, N + 3, (n,), generator=g, device="cuda", dtype=torch.int32)
        abi.hsa_qk_norm_rope(ctx, how, None, n, None, kc2, k_in=qkv[:, D:2 * D], pos=pos)
        ref, tol = _qk_ref(qkv[:, D:2 * D], wk, norm, 1e-5, H, d, table[pos.long()], layout)
        _within(kc2[:n], ref, tol)
        abi.hsa_sync_check(ctx)


def test_qk_norm_rope_of_zero_and_huge_rows():
    need_gpu()
    ctx = _ctx(4, 256, 2)
    q = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    q[1] = 1e18  # squares up to 1e36: the row's sum of 256 stays in fp32's range
    q[2, :3] = float("nan")
    q[3] = -2.0
    q0 = q.clone()
    abi.hsa_qk_norm_rope(ctx, abi.qk_rope(norm="row", eps=1e-6), None, 4, q)
    abi.hsa_sync_check(ctx)
    assert bool((q[0] == 0).all())
    assert bool(((q[1].float() - 1).abs() <= BF + 2.0 ** -14).all()) and bool(((q[3].float() + 1).abs() <= BF + 2.0 ** -14).all())
    assert bool(torch.isnan(q[2].float()).all())
    q = q0.clone()
    abi.hsa_qk_norm_rope(ctx, abi.qk_rope(norm="head", eps=1e-6), None, 4, q)
    assert bool(torch.isnan(q[2, :128].float()).all()) and bool((q[2, 128:] == 0).all())


def test_qk_norm_rope_reports_bad_rows():
    need_gpu()
    ctx = _ctx(6, 128, 1)
    g = _gen(2)
    qk = _randn(g, 4, 256, dtype=torch.bfloat16)
    table = _table(g, 5, 128)
    how = abi.qk_rope(norm="head", table=table, P=5, rot=128)

    def call(idx, in_place=False):
        kc, vc = torch.full((6, 128), 3.0, dtype=torch.bfloat16, device="cuda"), None
        q = torch.full((4, 128), 9.0, dtype=torch.bfloat16, device="cuda")
        i = torch.tensor(idx, dtype=torch.int32, device="cuda")
        abi.hsa_qk_norm_rope(ctx, how, i, 4, q, kc, q_in=qk[:, :128], k_in=None if in_place else qk[:, 128:])
        with pytest.raises(abi.HsaError) as e:
            abi.hsa_sync_check(ctx)
        assert e.value.status == 7
        return q, kc

    q, kc = call([0, -1, 6, 2])
    assert bool((q[1:3] == 0).all()) and not bool((q[0] == 0).all())
    assert bool((kc[[1, 3, 4, 5]] == 3.0).all()) and not bool((kc[0] == 3.0).all())
    q, kc = call([0, 1, 2, 5])       # cache row 5 is there, table row 5 is not
    assert bool((q[3] == 0).all()) and bool((kc[5] == 3.0).all())
    q, kc = call([0, 1, 1, 3], in_place=True)  # turned once, not twice
    once = torch.full((1, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    ref, tol = _qk_ref(once, None, "head", 1e-6, 1, 128, table[1:2], "half")
    _within(kc[1:2], ref, tol)


# ---------------------------------------------------------------- cross-attention

def _cross64(q, starts, k, v, lens, mask, H, Hk, d, scale):
    """Per sequence and head in 64 bits, unseen keys left out; also sum_j p_j |v_j|."""
    n = q.shape[0]
    o = torch.zeros(n, H, d, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(o)
    for b in range(len(starts) - 1):
        keys = torch.arange(lens[b], device="cuda")
        if mask is not None:
            keys = keys[mask[b, :lens[b]] != 0]
        if starts[b] >= starts[b + 1] or keys.numel() == 0:
            continue
        rows = slice(starts[b], starts[b + 1])
        for h in range(H):
            c = slice(h // (H // Hk) * d, (h // (H // Hk) + 1) * d)
            kk, vv = k[b, keys][:, c].double(), v[b, keys][:, c].double()
            p = torch.softmax(q[rows, h * d:(h + 1) * d].double() @ kk.t() * scale, dim=1)
            o[rows, h], mag[rows, h] = p @ vv, p @ vv.abs()
    return o.reshape(n, H * d), mag.reshape(n, H * d)


def _cross_tol(o, mag):
    """Each weight is rounded to bf16 once and the output once; scores are fp32
    sums of 128 products (their error, below 2^-10 of a weight, is the 1.3)."""
    return 1.3 * BF * (mag + o.abs())


def _cross_case(seed, H, Hk, d, starts, S, lens, holes, n=None, q_scale=2.0):
    g = _gen(seed)
    B, D = len(starts) - 1, H * d
    n = starts[-1] if n is None else n
    q = _randn(g, n, D, dtype=torch.bfloat16) * q_scale
    k, v = _randn(g, B, S, Hk * d, dtype=torch.bfloat16), _randn(g, B, S, Hk * d, dtype=torch.bfloat16)
    mask = (torch.rand(B, S, generator=g, device="cuda") > holes).to(torch.uint8) if holes else None
    return q, k, v, mask


@pytest.mark.parametrize("H,Hk,d,starts,S,lens,holes", [
    (1, 1, 128, [0, 1], 1, [1], 0),
    (2, 2, 64, [0, 1, 2, 3], 130, [130, 0, 1], 0),
    (2, 1, 128, [0, 300, 300, 301, 700], 257, [257, 5, 128, 129], 0),
    (12, 12, 128, [0, 513], 77, [77], 0),
    (4, 2, 64, [0, 255, 512], 512, [511, 300], 0.5),
    (3, 1, 128, [0, 2, 259], 700, [700, 640], 0.97),
    (1, 1, 128, [0] + list(range(1, 41)), 90, [90 - b for b in range(40)], 0.3),
    (2, 2, 64, [0, 1100], 4096, [4000], 0.1),
    (1, 1, 128, [0, 1], 5000, [5000], 0),
    (8, 2, 128, [0, 33, 66], 384, [384, 384], 0),
    (1, 1, 128, [0, 2, 4, 300], 5000, [5000, 0, 1], 0),        # key ranges of a sequence without keys
    (2, 1, 64, [0, 5, 9], 3000, [2999, 200], 0.995),           # ranges without a seen key
    (12, 12, 128, [0, 3000, 6111], 300, [300, 129], 0),        # several units a CTA
    (4, 4, 128, [0, 1, 2, 2, 3], 700, [700, 513, 9, 0], 0.3),  # single tokens, keys over a cluster
    (4, 1, 64, [0, 2, 4], 5000, [4999, 1], 0),                 # two queries x four heads a key head
    (12, 4, 128, [0] * 30 + [1, 20, 21], 130, [130 - b for b in range(32)], 0.1),  # one long one among short ones
    (4, 4, 64, [0, 8000, 8001, 20001], 333, [333, 333, 64], 0.2),
    (2, 2, 64, list(range(0, 4501, 3)), 40, [b % 41 for b in range(1500)], 0),  # more sequences than one search step
])
def test_cross_attention(H, Hk, d, starts, S, lens, holes):
    need_gpu()
    ctx = _ctx(1, H * d, H) if H * d % 128 == 0 else None
    q, k, v, mask = _cross_case(len(starts) + S, H, Hk, d, starts, S, lens, holes)
    B, n = len(lens), starts[-1]
    # what lies in unseen places must not matter
    seen = torch.arange(S, device="cuda")[None] < torch.tensor(lens, device="cuda")[:, None]
    if mask is not None:
        seen &= mask != 0
    k[~seen], v[~seen] = float("nan"), float("inf")
    o = torch.empty_like(q)
    st, ln = torch.tensor(starts, dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
    abi.hsa_cross_attention(ctx, q, st, n, B, k, v, S, o, kv_len=ln, kv_mask=mask, kv_heads=Hk)
    abi.hsa_sync_check(ctx)
    ref, mag = _cross64(q, starts, k, v, lens, mask, H, Hk, d, d ** -0.5)
    _within(o, ref, _cross_tol(ref, mag))
    for b in range(B):
        if not bool(seen[b].any()):
            assert bool((o[starts[b]:starts[b + 1]] == 0).all())
    again = torch.empty_like(q)
    abi.hsa_cross_attention(ctx, q, st, n, B, k, v, S, again, kv_len=ln,
                            kv_mask=None if mask is None else mask != 0, kv_heads=Hk)
    assert torch.equal(again, o)


def test_cross_attention_rows_of_no_sequence_are_left():
    need_gpu()
    ctx = _ctx(1, 128, 1)
    starts, lens = [300, 310, 600], [50, 40]
    q, k, v, _ = _cross_case(4, 1, 1, 128, starts, 64, lens, 0, n=900)
    o = torch.full_like(q, 6.0)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    abi.hsa_cross_attention(ctx, q, st, 900, 2, k, v, 64, o, kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    abi.hsa_sync_check(ctx)
    ref, mag = _cross64(q, starts, k, v, lens, None, 1, 1, 128, 128 ** -0.5)
    _within(o[300:600], ref[300:600], _cross_tol(ref, mag)[300:600])
    assert bool((o[:300] == 6.0).all()) and bool((o[600:] == 6.0).all())
    few = torch.full_like(q[:7], 6.0)  # the same with a few queries each
    st = torch.tensor([2, 3, 5], dtype=torch.int32, device="cuda")
    abi.hsa_cross_attention(ctx, q, st, 7, 2, k, v, 64, few, kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    abi.hsa_sync_check(ctx)
    ref, mag = _cross64(q[:7], [2, 3, 5], k, v, lens, None, 1, 1, 128, 128 ** -0.5)
    _within(few[2:5], ref[2:5], _cross_tol(ref, mag)[2:5])
    assert bool((few[:2] == 6.0).all()) and bool((few[5:] == 6.0).all())


@pytest.mark.parametrize("H,Hk,d,step,B,S,holes", [
    (24, 12, 64, 7, 40, 300, 0),    # two heads a tile row
    (12, 1, 128, 13, 20, 130, 0.2),
    (32, 4, 64, 16, 30, 513, 0),    # sequences that end with a tile
    (48, 3, 64, 2, 33, 900, 0.5),
    (32, 1, 64, 9, 32, 77, 0),
    (64, 1, 64, 40, 8, 1000, 0.9),  # more heads than are packed
    (32, 2, 128, 2, 8, 4096, 0),    # and key ranges that are merged
    (40, 8, 64, 3, 16, 300, 0),     # five heads a query, 125 of a tile's 128 rows
    (28, 4, 64, 17, 30, 200, 0.4),  # seven
    (20, 1, 64, 70, 3, 2500, 0),    # twenty, six queries a tile, merged key ranges
    (12, 4, 128, 33, 30, 140, 0.1),
    (24, 24, 64, 23, 13, 1389, 0),  # nothing to pack: a lone tile a unit
    (4, 4, 128, 120, 9, 700, 0.3),
])
def test_cross_attention_packs_the_heads_of_a_key_head(H, Hk, d, step, B, S, holes):
    need_gpu()
    ctx = _ctx(1, H * d, H)
    starts, lens = [5], []
    for b in range(B):  # one sequence without rows, some without keys, lengths around `step`
        starts.append(starts[-1] + (0 if b == 1 else step + (b % 3 - 1) * (step > 2)))
        lens.append(0 if b % 5 == 3 else S - 11 * b % S)
    n = starts[-1] + 3
    q, k, v, mask = _cross_case(H + S, H, Hk, d, starts, S, lens, holes, n=n)
    seen = torch.arange(S, device="cuda")[None] < torch.tensor(lens, device="cuda")[:, None]
    if mask is not None:
        seen &= mask != 0
    k[~seen], v[~seen] = float("nan"), float("inf")
    o = torch.full_like(q, 6.0)
    st, ln = torch.tensor(starts, dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
    abi.hsa_cross_attention(ctx, q, st, n, B, k, v, S, o, kv_len=ln, kv_mask=mask, kv_heads=Hk)
    abi.hsa_sync_check(ctx)
    ref, mag = _cross64(q, starts, k, v, lens, mask, H, Hk, d, d ** -0.5)
    rows = slice(starts[0], starts[-1])
    _within(o[rows], ref[rows], _cross_tol(ref, mag)[rows])
    assert bool((o[:5] == 6.0).all()) and bool((o[starts[-1]:] == 6.0).all())
    for b in range(B):
        if not bool(seen[b].any()):
            assert bool((o[starts[b]:starts[b + 1]] == 0).all())


def test_cross_attention_layouts_and_scale():
    """Keys and values as halves of one packed projection, sequence-major
    [S, B, ..] states, one sequence shared by all, a scale of the caller's."""
    need_gpu()
    H, d, S, B = 2, 128, 150, 3
    ctx = _ctx(1, H * d, H)
    starts = [0, 10, 300, 320]
    q, k, v, _ = _cross_case(9, H, H, d, starts, S, [S] * B, 0)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    o, want = torch.empty_like(q), torch.empty_like(q)
    abi.hsa_cross_attention(ctx, q, st, 320, B, k, v, S, want, scale=0.3)
    ref, mag = _cross64(q, starts, k, v, [S] * B, None, H, H, d, float(np.float32(0.3)))
    _within(want, ref, _cross_tol(ref, mag))
    kv = torch.cat([k, v], dim=2)
    abi.hsa_cross_attention(ctx, q, st, 320, B, kv[:, :, :H * d], kv[:, :, H * d:], S, o, scale=0.3)
    assert torch.equal(o, want)
    kt, vt = k.transpose(0, 1).contiguous().transpose(0, 1), v.transpose(0, 1).contiguous().transpose(0, 1)
    abi.hsa_cross_attention(ctx, q, st, 320, B, kt, vt, S, o, scale=0.3)
    assert torch.equal(o, want)
    # equal parts without offsets, for many queries and for few
    for n in (318, 6):
        e = torch.tensor([0, n // 3, 2 * n // 3, n], dtype=torch.int32, device="cuda")
        abi.hsa_cross_attention(ctx, q, e, n, B, k, v, S, want)
        abi.hsa_cross_attention(ctx, q, None, n, B, k, v, S, o)
        assert torch.equal(o[:n], want[:n])
    _refused(1, abi.hsa_cross_attention, ctx, q, None, 320, B, k, v, S, o)
    k1, v1 = k[:1].expand(B, S, H * d), v[:1].expand(B, S, H * d)
    abi.hsa_cross_attention(ctx, q, st, 320, B, k1, v1, S, o)
    abi.hsa_cross_attention(ctx, q, st, 320, B, k1.contiguous(), v1.contiguous(), S, want)
    assert torch.equal(o, want)
    abi.hsa_sync_check(ctx)


@pytest.mark.parametrize("n", [200, 40000])  # keys split over CTAs, and one CTA for all of a row's keys
def test_cross_attention_growing_scores(n):
    """Scores that rise by tens of powers of two per tile, behind a first tile
    that a mask empties: the running maximum has to move, more than once."""
    need_gpu()
    H, d, S = 1, 128, 900
    ctx = _ctx(1, d, H)
    g = _gen(8)
    q = torch.ones(n, d, dtype=torch.bfloat16, device="cuda")
    ramp = (torch.arange(S, device="cuda") * 2).float()
    k = (ramp[:, None] / 16).expand(S, d).to(torch.bfloat16)[None].contiguous()
    v = _randn(g, 1, S, d, dtype=torch.bfloat16)
    for sign in (1, -1):
        mask = torch.ones(1, S, dtype=torch.uint8, device="cuda")
        mask[0, 1:140] = 0
        mask[0, 500:640] = 0
        o = torch.empty_like(q)
        abi.hsa_cross_attention(ctx, q * sign, torch.tensor([0, n], dtype=torch.int32, device="cuda"), n, 1, k, v, S, o,
                                kv_mask=mask)
        abi.hsa_sync_check(ctx)
        ref, mag = _cross64(q * sign, [0, n], k, v, [S], mask, H, H, d, d ** -0.5)
        # scores reach 1300: fp32 holds them to 2^-13, a weight to 2^-12
        _within(o, ref, _cross_tol(ref, mag) + 2.0 ** -12 * mag)


def test_cross_attention_reports_bad_offsets_and_lengths():
    need_gpu()
    ctx = _ctx(1, 128, 1)
    q, k, v, _ = _cross_case(4, 1, 1, 128, [0, 100], 64, [64], 0)
    k, v = k.repeat(2, 1, 1), v.repeat(2, 1, 1)

    def status(starts, lens):
        o = torch.empty_like(q)
        abi.hsa_cross_attention(ctx, q, torch.tensor(starts, dtype=torch.int32, device="cuda"), 100, 2, k, v, 64, o,
                                kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        try:
            abi.hsa_sync_check(ctx)
            return 0
        except abi.HsaError as e:
            return e.status

    assert status([0, 50, 100], [64, 3]) == 0
    assert status([0, 50, 101], [64, 3]) == 7
    assert status([0, 70, 60], [64, 3]) == 7
    assert status([-5, 70, 80], [64, 3]) == 7
    assert status([0, 50, 100], [65, 3]) == 7
    assert status([0, 50, 100], [64, -1]) == 7
    assert status([0, 50, 100], [64, 64]) == 0


# ---------------------------------------------------------------- streams, graphs, together

def test_operators_on_another_stream_and_in_a_graph():
    """Captured once, replayed with other inputs and other lengths: a graph
    reads what is there at the replay."""
    need_gpu()
    side = torch.cuda.Stream()
    N, H, d, S = 300, 2, 128, 200
    D = H * d
    ctx = _ctx(N, D, H, stream=side)
    g = _gen(21)
    idx = torch.arange(0, N, 2, dtype=torch.int32, device="cuda")
    n = idx.numel()
    x = _randn(g, n, D, dtype=torch.bfloat16)
    w = torch.randint(-127, 128, (3 * D, D), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.full((3 * D,), 1e-3, device="cuda")
    table = torch.empty(N, d // 2, 2, device="cuda")
    xq, xs = torch.empty(n, D, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    qkv, q = torch.empty(n, 3 * D, dtype=torch.bfloat16, device="cuda"), torch.empty(n, D, dtype=torch.bfloat16, device="cuda")
    kc, vc = torch.zeros(N, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(N, D, dtype=torch.bfloat16, device="cuda")
    kt, vt = _randn(g, 2, S, D, dtype=torch.bfloat16), _randn(g, 2, S, D, dtype=torch.bfloat16)
    st = torch.tensor([0, 70, n], dtype=torch.int32, device="cuda")
    ln = torch.tensor([200, 33], dtype=torch.int32, device="cuda")
    o = torch.empty_like(q)
    cfg = abi.rope_cfg([d])
    how = abi.qk_rope(norm="head", table=table, P=N, rot=d)

    def chain():
        abi.hsa_rope_table(ctx, cfg, None, N, table)
        abi.hsa_quant_rows(ctx, x, n, D, xq, xs)
        abi.hsa_linear_quant(ctx, xq, xs, n, D, w, sw, 3 * D, qkv)
        abi.hsa_qk_norm_rope(ctx, how, idx, n, q, kc, vc, q_in=qkv[:, :D], k_in=qkv[:, D:2 * D], v_in=qkv[:, 2 * D:])
        abi.hsa_cross_attention(ctx, q, st, n, 2, kt, vt, S, o, kv_len=ln)

    torch.cuda.synchronize()
    chain()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        chain()
    x.copy_(_randn(g, n, D, dtype=torch.bfloat16))
    ln.copy_(torch.tensor([7, 190]))
    st.copy_(torch.tensor([0, 100, n]))
    torch.cuda.synchronize()
    outs = []
    for f in (graph.replay, chain):
        for t in (q, kc, vc, o):
            t.zero_()
        torch.cuda.synchronize()
        f()
        torch.cuda.synchronize()
        outs.append([t.clone() for t in (q, kc, vc, o)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    abi.hsa_sync_check(ctx)
    ref, mag = _cross64(outs[0][0], [0, 100, n], kt, vt, [7, 190], None, H, H, d, d ** -0.5)
    _within(outs[0][3], ref, _cross_tol(ref, mag))
    del graph


def test_two_contexts_at_once():
    """Two contexts on two streams have scratch of their own: their calls may overlap."""
    need_gpu()
    H, d, S = 2, 128, 3000
    D = H * d
    g = _gen(31)
    q = _randn(g, 300, D, dtype=torch.bfloat16)
    k, v = _randn(g, 1, S, D, dtype=torch.bfloat16), _randn(g, 1, S, D, dtype=torch.bfloat16)
    w = torch.randint(-127, 128, (700, D), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.ones(700, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = []
    for s in streams:
        ctx = _ctx(1, D, H, stream=s)
        runs.append((ctx, torch.empty_like(q), torch.empty(300, D, dtype=torch.int8, device="cuda"), torch.empty(300, device="cuda"),
                     torch.empty(300, 700, dtype=torch.bfloat16, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for ctx, o, q8, s8, y in runs:
            abi.hsa_cross_attention(ctx, q, None, 300, 1, k, v, S, o)  # split over keys: partial results in scratch
            abi.hsa_quant_rows(ctx, o, 300, D, q8, s8)
            abi.hsa_linear_quant(ctx, q8, s8, 300, D, w, sw, 700, y)
    for ctx, *_ in runs:
        abi.hsa_sync_check(ctx)
    ref, mag = _cross64(q, [0, 300], k, v, [S], None, H, H, d, d ** -0.5)
    for ctx, o, q8, s8, y in runs:
        _within(o, ref, _cross_tol(ref, mag))
        assert torch.equal(o, runs[0][1]) and torch.equal(y, runs[0][4])


def test_no_rows_launch_nothing():
    need_gpu()
    ctx = _ctx(4, 128, 1)
    before = abi.hsa_kernel_launches(ctx)
    b, f, i8 = (torch.zeros(4, 128, dtype=t, device="cuda") for t in (torch.bfloat16, torch.float32, torch.int8))
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    abi.hsa_quant_rows(ctx, b, 0, 128, i8, f)
    abi.hsa_linear_quant(ctx, i8, f, 0, 128, i8, f, 4, b)
    abi.hsa_ln_gather_quant(ctx, f, i, 0, i8, f)
    abi.hsa_rope_table(ctx, abi.rope_cfg([128]), None, 0, f)
    abi.hsa_rope(ctx, b, 0, 1, f, 4, 128, b)
    abi.hsa_qk_norm_rope(ctx, abi.qk_rope(), i, 0, b, b)
    abi.hsa_cross_attention(ctx, b, i, 0, 1, b[None], b[None], 4, b)
    assert abi.hsa_kernel_launches(ctx) == before
    abi.hsa_sync_check(ctx)


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: their first and last rows."""
    need_gpu()
    g = _gen(6)
    N, H, d = 420000, 40, 128
    D = H * d  # N * D = 2.15e9
    ctx = _ctx(N, D, H)
    idx = torch.tensor([0, 1, N - 2, N - 1], dtype=torch.int32, device="cuda")
    rows = idx.long()
    big = torch.zeros(N, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(N, D, dtype=torch.bfloat16, device="cuda")
    few = _randn(g, 4, D, dtype=torch.bfloat16)
    table = _table(g, N, 32)
    # cache rows
    abi.hsa_qk_norm_rope(ctx, abi.qk_rope(table=table, P=N, rot=32), idx, 4, None, big, k_in=few)
    ref, tol = _qk_ref(few, None, "head", 1e-6, H, d, table[rows], "half")
    _within(big[rows], ref, tol)
    # rotated rows
    abi.hsa_rope(ctx, big, N, H, table, N, 32, out)
    ref, mag = _turned(big[rows].double().view(4, H, d), table[rows].double(), "half")
    _within(out[rows].view(4, H, d), ref, BF * ref.abs() + 4 * F32 * mag)
    # queries and outputs
    big[rows] = few
    k, v = _randn(g, 1, 5, D, dtype=torch.bfloat16), _randn(g, 1, 5, D, dtype=torch.bfloat16)
    abi.hsa_cross_attention(ctx, big, None, N, 1, k, v, 5, out)
    ref, mag = _cross64(few, [0, 4], k, v, [5], None, H, H, d, d ** -0.5)
    _within(out[rows], ref, _cross_tol(ref, mag))
    # keys far down a cache that all sequences share
    kv = big.view(1, N, D)
    st, ln = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([N], dtype=torch.int32, device="cuda")
    mask = torch.zeros(1, N, dtype=torch.uint8, device="cuda")
    mask[0, rows] = 1
    for n, start in ((1, st), (300, None)):
        q = _randn(g, n, D, dtype=torch.bfloat16)
        o = torch.empty_like(q)
        abi.hsa_cross_attention(ctx, q, start, n, 1, kv, kv, N, o, kv_len=ln, kv_mask=mask)
        ref, mag = _cross64(q, [0, n], few[None], few[None], [4], None, H, H, d, d ** -0.5)
        _within(o, ref, _cross_tol(ref, mag))
    # quantised rows, and a product with more than 2^31 outputs
    q8 = out.view(torch.int8).view(-1)[:N * D].view(N, D)
    s = torch.empty(N, device="cuda")
    abi.hsa_quant_rows(ctx, big, N, D, q8, s)
    want_q, want_s = _quantised(few)
    assert (q8[rows].cpu().numpy() == want_q).all() and (s[rows].cpu().numpy() == want_s).all()
    assert bool((s[2:-2] == 0).all())
    w, sw = torch.randint(-127, 128, (D, 64), generator=g, device="cuda", dtype=torch.int8), torch.ones(D, device="cuda")
    a = torch.randint(-127, 128, (N, 64), generator=g, device="cuda", dtype=torch.int8)
    s.fill_(1.0)
    abi.hsa_linear_quant(ctx, a, s, N, 64, w, sw, D, out)
    ref = a[rows].double() @ w.double().t()
    _within(out[rows], ref, (BF + 4 * F32) * ref.abs())
    abi.hsa_sync_check(ctx)


# ---------------------------------------------------------------- refusals

def _refused(status, f, *a, **kw):
    with pytest.raises(abi.HsaError) as e:
        f(*a, **kw)
    assert e.value.status == status and str(e.value)


def test_refusals():
    need_gpu()
    ctx = _ctx(8, 256, 2)
    lib, P = abi.load(), ctx.ptr
    b = torch.zeros(8, 512, dtype=torch.bfloat16, device="cuda")
    f = torch.zeros(8, 512, device="cuda")
    i8 = torch.zeros(8, 512, dtype=torch.int8, device="cuda")
    i = torch.zeros(16, dtype=torch.int32, device="cuda")
    u8 = torch.zeros(8, 512, dtype=torch.uint8, device="cuda")
    ARG, SHAPE = 1, 3
    before = abi.hsa_kernel_launches(ctx)
    a = lambda t: t.data_ptr()  # noqa: E731
    for st, args in [(ARG, (a(b), 2, 8, 64, 512, a(i8), 512, a(f))), (SHAPE, (a(b), 0, 8, 0, 512, a(i8), 512, a(f))),
                     (SHAPE, (a(b), 0, 8, 131072, 131072, a(i8), 131072, a(f))), (SHAPE, (a(b), 0, 8, 64, 63, a(i8), 512, a(f))),
                     (SHAPE, (a(b), 0, 8, 64, 512, a(i8), 72, a(f))), (SHAPE, (a(b), 0, -1, 64, 512, a(i8), 64, a(f))),
                     (ARG, (None, 0, 8, 64, 512, a(i8), 64, a(f))), (ARG, (a(b) + 2, 0, 8, 64, 512, a(i8), 64, a(f)))]:
        assert lib.hsa_quant_rows(P, *args) == st
    for st, args in [(SHAPE, (a(i8), 512, a(f), 8, 0, a(i8), 512, a(f), 8, a(b))), (SHAPE, (a(i8), 512, a(f), 8, 64, a(i8), 512, a(f), 0, a(b))),
                     (SHAPE, (a(i8), 56, a(f), 8, 64, a(i8), 512, a(f), 8, a(b))), (SHAPE, (a(i8), 72, a(f), 8, 64, a(i8), 512, a(f), 8, a(b))),
                     (SHAPE, (a(i8), 512, a(f), 8, 131072, a(i8), 512, a(f), 8, a(b))), (ARG, (a(i8), 512, None, 8, 64, a(i8), 512, a(f), 8, a(b))),
                     (ARG, (a(i8), 512, a(f), 8, 64, a(i8) + 8, 512, a(f), 8, a(b)))]:
        assert lib.hsa_linear_quant(P, *args) == st
    _refused(ARG, abi.hsa_ln_gather_quant, ctx, f.view(-1)[:2048], i, 9, i8.view(-1), f.view(-1))
    _refused(ARG, abi.hsa_ln_gather_quant, ctx, f, i, 8, i8, f, shift=f)
    wide = abi.hsa_create(N=1, D=5248, H=41, F=64, L=0, T=1, budgets=[1], counts=[1])
    _refused(SHAPE, abi.hsa_ln_gather_quant, wide, torch.zeros(5248, device="cuda"), i, 1,
             torch.zeros(5248, dtype=torch.int8, device="cuda"), f)
    for st, cfg in [(SHAPE, abi.rope_cfg([63])), (SHAPE, abi.rope_cfg([0])), (SHAPE, abi.rope_cfg([128, 2])), (ARG, abi.rope_cfg([64], base=1.0)),
                    (ARG, abi.rope_cfg([64], base=float("nan"))), (ARG, abi.rope_cfg([64], scaling="linear", factor=0.5)),
                    (ARG, abi.rope_cfg([64], scaling="parts", factor=2.0)), (ARG, abi.rope_cfg([64], scaling="parts", factor=2.0, orig_len=9.0, fast=1.0)),
                    (ARG, abi.rope_cfg([64], amp=float("inf"))), (ARG, abi.rope_cfg([32, 32]))]:
        _refused(st, abi.hsa_rope_table, ctx, cfg, None, 1, torch.zeros(256, device="cuda"))
    _refused(ARG, abi.hsa_rope_table, ctx, abi.rope_cfg([64]), None, -1, f)
    for rot in (0, 8, 40, 144):
        _refused(SHAPE, abi.hsa_rope, ctx, b, 2, 2, f, 2, rot, b)
    _refused(SHAPE, abi.hsa_rope, ctx, b, 2, 0, f, 2, 128, b)
    _refused(SHAPE, abi.hsa_rope, ctx, b.view(-1)[:8 * 260].view(8, 260), 2, 2, f, 2, 128, b)
    _refused(ARG, abi.hsa_rope, ctx, b, 3, 2, f, 2, 128, b)
    assert lib.hsa_rope(P, a(b), 512, 0, 2, 2, a(f), 2, 128, None, 2, 0, a(b), 512) == ARG
    assert lib.hsa_rope(P, a(b), 512, 3, 2, 2, a(f), 2, 128, None, 0, 0, a(b), 512) == ARG
    q = torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")
    how = abi.qk_rope()
    _refused(ARG, abi.hsa_qk_norm_rope, ctx, how, i, 8, None, None)
    _refused(ARG, abi.hsa_qk_norm_rope, ctx, how, i, 8, q, v_cache=q)
    _refused(ARG, abi.hsa_qk_norm_rope, ctx, how, i, 8, None, q, q_in=b)
    _refused(ARG, abi.hsa_qk_norm_rope, ctx, abi.qk_rope(eps=-1.0), i, 8, q)
    _refused(SHAPE, abi.hsa_qk_norm_rope, ctx, abi.qk_rope(table=f, P=2, rot=24), i, 8, q)
    assert lib.hsa_qk_norm_rope(P, None, a(i), None, 8, None, 0, a(q), None, 0, None, None, 0, None) == ARG
    assert lib.hsa_qk_norm_rope(P, how, a(i), None, 9, None, 0, a(q), None, 0, None, None, 0, None) == ARG
    assert lib.hsa_qk_norm_rope(P, how, a(i), None, 8, a(b), 250, a(q), None, 0, None, None, 0, None) == SHAPE
    k = torch.zeros(2, 4, 256, dtype=torch.bfloat16, device="cuda")
    for st, kw in [(SHAPE, dict(kv_heads=0)), (ARG, dict(scale=-1.0)), (ARG, dict(scale=float("nan")))]:
        _refused(st, abi.hsa_cross_attention, ctx, q, i, 8, 2, k, k, 4, q, **kw)
    k3 = torch.zeros(2, 4, 384, dtype=torch.bfloat16, device="cuda")
    _refused(SHAPE, abi.hsa_cross_attention, ctx, q, i, 8, 2, k3, k3, 4, q, kv_heads=3)
    odd = torch.zeros(2, 4, 260, dtype=torch.bfloat16, device="cuda")[:, :, :256]
    _refused(SHAPE, abi.hsa_cross_attention, ctx, q, i, 8, 2, odd, odd, 4, q)
    # on the Python side: types, sizes and strides before anything reaches the library
    for f_bad in (lambda: abi.hsa_quant_rows(ctx, i8, 8, 64, i8, f), lambda: abi.hsa_quant_rows(ctx, b.t(), 8, 8, i8, f),
                  lambda: abi.hsa_linear_quant(ctx, i8, f, 8, 512, i8, f, 8, b.view(-1)[:63]),
                  lambda: abi.hsa_linear_quant(ctx, u8, f, 8, 512, i8, f, 8, b), lambda: abi.hsa_rope(ctx, b, 8, 5, f, 8, 128, b),
                  lambda: abi.hsa_rope(ctx, b, 8, 2, f, 8, 128, f), lambda: abi.hsa_rope(ctx, b, 9, 2, f, 9, 128, b),
                  lambda: abi.hsa_cross_attention(ctx, q, i[:2], 8, 2, k, k, 4, q), lambda: abi.hsa_cross_attention(ctx, q, i, 8, 2, k[:1], k, 4, q),
                  lambda: abi.hsa_cross_attention(ctx, q, i, 8, 2, k, k, 4, q, kv_mask=u8[:1, :7])):
        with pytest.raises(ValueError):
            f_bad()
    assert abi.hsa_kernel_launches(ctx) == before
    abi.hsa_sync_check(ctx)
