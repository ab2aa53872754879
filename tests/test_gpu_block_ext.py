"""The block with rotary positions, query/key norms, masked text and 8-bit
weights (hsa_layer_forward_ext, hsa_step_ext), on the active set.

Stage by stage it is the public calls it names, bit for bit; as a whole it is
compared with a 64-bit implementation within the bf16 tolerance of the plain
block's tests (1e-2 of the largest increment).
"""

import pytest

from gpu_util import BF16_TOL, bf, dev, host, need_gpu, normwise, torch
from token_sparse_denoising_layer_b200 import abi, synth
from token_sparse_denoising_layer_b200.loop import HsaLoop

pytestmark = pytest.mark.gpu

_KEYS = ("w_qkv", "w_o", "w_1", "w_2")


class Case:
    """Seeded inputs of one block on the device."""

    def __init__(self, N, D, H, F, a, n_txt, seed, norm="head", layout="half", rot=None):
        self.N, self.D, self.H, self.F, self.a, self.n_txt, self.d = N, D, H, F, a, n_txt, D // H
        self.norm, self.layout = norm, layout
        self.ctx = abi.hsa_create(N=N, D=D, H=H, F=F, L=1, T=1, budgets=[1], counts=[N])
        w = synth.layer_weights(D, F, seed)
        self.w = [bf(w[k]) for k in _KEYS]
        self.lw = abi.layer_weights(*self.w)
        self.x = dev(synth.hidden_rows(N, D, seed))
        ks, vs = synth.stale_kv(N, D, seed)
        self.kc, self.vc = bf(ks), bf(vs)
        self.idx = dev(synth.random_active_set(N, a, seed))
        self.mod = dev(synth.modulation(D, seed))
        cross = synth.cross_attention_weights(D, n_txt, seed)
        self.cross = {k: bf(v) for k, v in cross.items()}
        self.xa = abi.cross_attn(self.cross["w_q"], self.cross["w_o"], self.cross["k_txt"],
                                 self.cross["v_txt"], n_txt)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rot = self.d if rot is None else rot
        width = D if norm == "row" else self.d
        self.w_q, self.w_k = (1 + 0.1 * torch.randn(width, generator=g, device="cuda") for _ in range(2))
        self.table = torch.empty(N, self.rot // 2, 2, device="cuda")
        abi.hsa_rope_table(self.ctx, abi.rope_cfg([self.rot]), None, N, self.table)
        self.qk = abi.qk_rope(norm=norm, w_q=self.w_q, w_k=self.w_k, eps=1e-6, table=self.table, P=N, rot=self.rot,
                              layout=layout)
        self.mask = (torch.rand(n_txt, generator=g, device="cuda") > 0.3).to(torch.uint8)
        self.txt_len = torch.tensor([max(1, n_txt - 5)], dtype=torch.int32, device="cuda")

    def state(self):
        return self.x.clone(), self.kc.clone(), self.vc.clone()

    def run(self, ext, w=True):
        x, kc, vc = self.state()
        abi.hsa_layer_forward_ext(self.ctx, self.lw if w else None, ext, x, self.idx, self.a, kc, vc)
        abi.hsa_sync_check(self.ctx)
        return x, kc, vc


def _same(a, b):
    return all(torch.equal(s, t) for s, t in zip(a, b))


def test_without_extensions_it_is_the_plain_and_the_conditioned_block():
    need_gpu()
    c = Case(700, 256, 2, 512, 333, 77, 3)
    plain = c.state()
    abi.hsa_layer_forward(c.ctx, c.lw, plain[0], c.idx, c.a, plain[1], plain[2])
    assert _same(c.run(None), plain) and _same(c.run(abi.block_ext()), plain)
    cond = c.state()
    abi.hsa_layer_forward_cond(c.ctx, c.lw, c.mod, c.xa, cond[0], c.idx, c.a, cond[1], cond[2])
    assert _same(c.run(abi.block_ext(mod=c.mod, xa=c.xa)), cond)


def _cross_stage(c, x, txt_len, mask):
    u, q, o = (torch.empty(c.a, c.D, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    abi.hsa_ln_gather(c.ctx, x, c.idx, c.a, u)
    abi.hsa_linear(c.ctx, u, c.a, c.D, c.cross["w_q"], c.D, q)
    abi.hsa_cross_attention(c.ctx, q, None, c.a, 1, c.cross["k_txt"][None], c.cross["v_txt"][None], c.n_txt, o,
                            kv_len=txt_len, kv_mask=mask)
    abi.hsa_out_proj_residual(c.ctx, c.cross["w_o"], o, c.idx, c.a, x)


@pytest.mark.parametrize("args,kw", [
    ((700, 256, 2, 512, 333, 77), dict(norm="head", layout="half")),
    ((300, 128, 2, 256, 300, 1), dict(norm="row", layout="interleaved", rot=32)),
    ((1500, 1536, 12, 6144, 260, 512), dict(norm="row", layout="interleaved")),
    ((513, 640, 5, 128, 1, 200), dict(norm="none", layout="half")),
])
def test_bf16_block_is_its_stages_and_near_64_bits(args, kw):
    need_gpu()
    c = Case(*args, seed=7, **kw)
    got = c.run(abi.block_ext(mod=c.mod, xa=c.xa, txt_len=c.txt_len, txt_mask=c.mask, qk=c.qk))
    x, kc, vc = c.state()
    u, q, o = (torch.empty(c.a, c.D, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    abi.hsa_ln_gather_mod(c.ctx, x, c.idx, c.a, u, c.mod[0], c.mod[1])
    abi.hsa_qkv_project(c.ctx, c.w[0], u, c.idx, c.a, q, kc, vc)
    abi.hsa_qk_norm_rope(c.ctx, c.qk, c.idx, c.a, q, kc)
    abi.hsa_attention(c.ctx, q, c.a, kc, vc, o)
    abi.hsa_out_proj_residual_gated(c.ctx, c.w[1], o, c.idx, c.a, x, c.mod[2])
    _cross_stage(c, x, c.txt_len, c.mask)
    abi.hsa_mlp_residual_mod(c.ctx, c.w[2], c.w[3], x, c.idx, c.a, c.mod[3], c.mod[4], c.mod[5])
    abi.hsa_sync_check(c.ctx)
    assert _same(got, (x, kc, vc))
    # the whole block in 64 bits
    rows = c.idx.long()
    ref, k64, v64 = _block64(c)
    rest = torch.ones(c.N, dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert torch.equal(got[0][rest], c.x[rest]) and torch.equal(got[1][rest], c.kc[rest])
    assert normwise(host((got[0] - c.x)[rows]), (ref - c.x.double())[rows].cpu().numpy()) <= BF16_TOL
    assert normwise(host(got[1][rows]), k64[rows].cpu().numpy()) <= BF16_TOL
    assert normwise(host(got[2][rows]), v64[rows].cpu().numpy()) <= BF16_TOL


def _ln64(x):
    return (x - x.mean(1, keepdim=True)) / torch.sqrt(x.var(1, unbiased=False, keepdim=True) + 1e-5)


def _heads64(y, w, c):
    """Norm and rotation of [n, D] rows at the active tokens' places."""
    n, H, d = y.shape[0], c.H, c.d
    if c.norm == "row":
        y = y / torch.sqrt((y * y).mean(1, keepdim=True) + 1e-6) * w.double()
    y = y.reshape(n, H, d)
    if c.norm == "head":
        y = y / torch.sqrt((y * y).mean(2, keepdim=True) + 1e-6) * w.double()
    half = c.rot // 2
    f = 10000.0 ** (-2.0 * torch.arange(half, dtype=torch.float64, device="cuda") / c.rot)
    ang = c.idx.double()[:, None] * f
    cos, sin = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    out = y.clone()
    i = (slice(0, half), slice(half, c.rot)) if c.layout == "half" else (slice(0, c.rot, 2), slice(1, c.rot, 2))
    a, b = y[..., i[0]], y[..., i[1]]
    out[..., i[0]], out[..., i[1]] = a * cos - b * sin, b * cos + a * sin
    return out.reshape(n, H * d)


def _attend64(q, k, v, H):
    d = q.shape[1] // H
    out = []
    for h in range(H):
        s = slice(h * d, (h + 1) * d)
        out.append(torch.softmax(q[:, s] @ k[:, s].t() / d ** 0.5, dim=1) @ v[:, s])
    return torch.cat(out, dim=1)


def _block64(c):
    rows, D = c.idx.long(), c.D
    w_qkv, w_o, w_1, w_2 = (w.double() for w in c.w)
    x, k, v, m = c.x.double().clone(), c.kc.double().clone(), c.vc.double().clone(), c.mod.double()
    u = _ln64(x[rows]) * (1 + m[1]) + m[0]
    qkv = u @ w_qkv.t()
    q = _heads64(qkv[:, :D], c.w_q, c)
    k[rows], v[rows] = _heads64(qkv[:, D:2 * D], c.w_k, c), qkv[:, 2 * D:]
    x[rows] += m[2] * (_attend64(q, k, v, c.H) @ w_o.t())
    seen = torch.nonzero(c.mask[:int(c.txt_len)]).flatten()
    if seen.numel():
        o = _attend64(_ln64(x[rows]) @ c.cross["w_q"].double().t(), c.cross["k_txt"].double()[seen],
                      c.cross["v_txt"].double()[seen], c.H)
        x[rows] += o @ c.cross["w_o"].double().t()
    u = _ln64(x[rows]) * (1 + m[4]) + m[3]
    h = torch.nn.functional.gelu(u @ w_1.t())
    x[rows] += m[5] * (h @ w_2.t())
    return x, k, v


def _product(aq, sa, wq, sw):
    """The 8-bit product before its epilogue: exact sums, then fp32 scales in the kernel's order."""
    acc = (aq.double() @ wq.double().t()).float()  # below 2^53 exactly; one rounding to fp32
    return acc * sa[:, None] * sw[None, :]


@pytest.mark.parametrize("args,gated", [((700, 256, 2, 512, 333, 77), True), ((300, 128, 2, 192, 300, 9), False),
                                        ((2100, 1536, 12, 6144, 1030, 512), True), ((64, 512, 4, 8960, 5, 40), True)])
def test_8bit_block_is_its_stages(args, gated):
    need_gpu()
    c = Case(*args, seed=11)
    wq = abi.layer_weights_quant(c.ctx, *c.w)
    mod = c.mod if gated else None
    got = c.run(abi.block_ext(mod=mod, xa=c.xa, txt_len=c.txt_len, qk=c.qk, wq=wq), w=False)
    (w_qkv, s_qkv), (w_o, s_o), (w_1, s_1), (w_2, s_2) = wq._keep
    x, kc, vc = c.state()
    rows, D, a = c.idx.long(), c.D, c.a
    row = lambda r: None if mod is None else mod[r]  # noqa: E731
    uq, us = torch.empty(a, D, dtype=torch.int8, device="cuda"), torch.empty(a, device="cuda")
    abi.hsa_ln_gather_quant(c.ctx, x, c.idx, a, uq, us, row(0), row(1))
    qkv = torch.empty(a, 3 * D, dtype=torch.bfloat16, device="cuda")
    abi.hsa_linear_quant(c.ctx, uq, us, a, D, w_qkv, s_qkv, 3 * D, qkv)
    assert torch.equal(qkv, _product(uq, us, w_qkv, s_qkv).to(torch.bfloat16))
    q, o = qkv[:, :D].contiguous(), torch.empty(a, D, dtype=torch.bfloat16, device="cuda")
    abi.hsa_qk_norm_rope(c.ctx, c.qk, c.idx, a, q, kc, vc, k_in=qkv[:, D:2 * D], v_in=qkv[:, 2 * D:])
    abi.hsa_attention(c.ctx, q, a, kc, vc, o)
    abi.hsa_quant_rows(c.ctx, o, a, D, uq, us)
    y = _product(uq, us, w_o, s_o)
    x[rows] += y if mod is None else mod[2] * y
    _cross_stage(c, x, c.txt_len, None)
    before_mlp = x.clone()
    abi.hsa_ln_gather_quant(c.ctx, x, c.idx, a, uq, us, row(3), row(4))
    h = torch.nn.functional.gelu(_product(uq, us, w_1, s_1).double()).to(torch.bfloat16)
    hq, hs = torch.empty(a, c.F, dtype=torch.int8, device="cuda"), torch.empty(a, device="cuda")
    abi.hsa_quant_rows(c.ctx, h, a, c.F, hq, hs)
    y = _product(hq, hs, w_2, s_2)
    x[rows] += y if mod is None else mod[5] * y
    abi.hsa_sync_check(c.ctx)
    assert _same(got[1:], (kc, vc))
    # The MLP's GELU may differ from the 64-bit one by a bf16 step, so a few
    # hidden bytes by one: were every byte rounded anew, the product would move by
    # about 1e-2 of its size (1/127 of the top, sqrt(2/12) of a step, top about 4
    # deviations); all else is exact.
    assert normwise(host((got[0] - before_mlp)[rows]), host((x - before_mlp)[rows])) <= 1e-2
    rest = torch.ones(c.N, dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert torch.equal(got[0][rest], c.x[rest])


def _ext_loop(quant):
    spec = synth.WORKLOADS["tiny_dit"]
    sh, T = spec["shape"], spec["T"]
    counts = synth.group_counts(sh.N, spec["fractions"])
    w = synth.model_weights(sh, 5)
    layers = [tuple(bf(lw[k]) for k in _KEYS) for lw in w["layers"]]
    loop = HsaLoop(sh.N, sh.D, sh.H, sh.F, layers, dev(w["w_in"]), dev(w["w_head"]), T, spec["budgets"], counts,
                   shift=spec["shift"])
    d = sh.D // sh.H
    # frame, row and column of each token of the 4 x 8 x 8 latent
    n = torch.arange(sh.N, device="cuda")
    pos = torch.stack([n // 64, n // 8 % 8, n % 8], dim=1).to(torch.int32).contiguous()
    table = torch.empty(sh.N, d // 2, 2, device="cuda")
    abi.hsa_rope_table(loop.ctx, abi.rope_cfg([d - 2 * (d // 3 // 2 * 2), d // 3 // 2 * 2, d // 3 // 2 * 2]), pos, sh.N, table)
    exts = []
    txt_len = torch.tensor([20], dtype=torch.int32, device="cuda")
    for l, lw in enumerate(layers):
        cr = {k: bf(v) for k, v in synth.cross_attention_weights(sh.D, 33, l).items()}
        exts.append(abi.block_ext(mod=dev(synth.modulation(sh.D, l)), xa=abi.cross_attn(cr["w_q"], cr["w_o"], cr["k_txt"], cr["v_txt"], 33),
                                  txt_len=txt_len, qk=abi.qk_rope(norm="head", table=table, P=sh.N, rot=d),
                                  wq=abi.layer_weights_quant(loop.ctx, *lw) if quant else None))
    return loop, abi.StepExt(exts), txt_len, synth.latent(sh.N, 16, 5), synth.random_split(sh.N, counts, 5), counts


@pytest.mark.parametrize("quant", [False, True])
def test_loop_with_extensions_replays_as_one_graph_with_another_prompt_length(quant):
    need_gpu()
    loop, ext, txt_len, x0, g0, counts = _ext_loop(quant)
    xs = []
    for length in (20, 33, 20):
        txt_len.fill_(length)
        loop.reset(x0, g0)
        loop.run(ext=ext)
        abi.hsa_sync_check(loop.ctx)
        xs.append(host(loop.x))
    assert (xs[0] == xs[2]).all() and not (xs[0] == xs[1]).all() and abs(xs[0]).max() < 1e3
    assert [int((host(loop.g) == k).sum()) for k in range(2)] == counts
    loop.capture(ext=ext)
    for length, want in ((33, xs[1]), (20, xs[0])):
        txt_len.fill_(length)
        loop.reset(x0, g0)
        loop.replay()
        abi.hsa_sync_check(loop.ctx)
        assert (host(loop.x) == want).all()
    loop.close()


def test_refusals():
    need_gpu()
    c = Case(64, 128, 1, 64, 8, 4, 1)

    def refused(status, ext, w=True):
        x, kc, vc = c.state()
        with pytest.raises(abi.HsaError) as e:
            abi.hsa_layer_forward_ext(c.ctx, c.lw if w else None, ext, x, c.idx, c.a, kc, vc)
        assert e.value.status == status and str(e.value)
        assert torch.equal(x, c.x)

    refused(1, None, w=False)
    refused(1, abi.block_ext(txt_len=c.txt_len))
    wq = abi.layer_weights_quant(c.ctx, *c.w)
    wq.s_1 = None
    refused(1, abi.block_ext(wq=wq))
    bad = abi.cross_attn(c.cross["w_q"], c.cross["w_o"], c.cross["k_txt"], c.cross["v_txt"], 0)
    refused(3, abi.block_ext(xa=bad))
    wide = abi.hsa_create(N=1, D=5248, H=41, F=64, L=0, T=1, budgets=[1], counts=[1])
    one = torch.zeros(5248, device="cuda")
    need = abi.block_ext(wq=abi.layer_weights_quant(c.ctx, *c.w))
    with pytest.raises(ValueError):  # another shape's weights
        abi.hsa_layer_forward_ext(wide, None, need, one, c.idx, 1, one, one)
    assert abi.load().hsa_layer_forward_ext(wide.ptr, None, need, one.data_ptr(), c.idx.data_ptr(), 1, one.data_ptr(),
                                            one.data_ptr()) == 3
    for ext in (abi.block_ext(mod=c.mod[:5].contiguous()), abi.block_ext(qk=abi.qk_rope(table=c.table, P=c.N - 1, rot=c.rot)),
                abi.block_ext(qk=abi.qk_rope(norm="row", w_q=c.w_q[:64]))):
        with pytest.raises(ValueError):
            x, kc, vc = c.state()
            abi.hsa_layer_forward_ext(c.ctx, c.lw, ext, x, c.idx, c.a, kc, vc)
    with pytest.raises(ValueError):
        abi.block_ext(xa=c.xa, txt_mask=c.mask[:1])
    loop, ext, _, _, _, _ = _ext_loop(False)
    with pytest.raises(ValueError):
        loop.step(0, cond=abi.StepCond(), ext=ext)
    with pytest.raises(ValueError):
        loop.step(0, ext=abi.StepExt([abi.block_ext()]))
    loop.close()
