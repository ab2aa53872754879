"""The operators of a quantised, rotary, text-conditioned transformer block, as cases that can be timed.

Four operators that stand around the active-row products of the denoising step:

  q8     rows quantised to 8-bit integers with a scale each, times a weight kept in 8-bit integers with a scale per output channel
  rope   rotary positions: the table of cosines and sines (several axes, long-context scalings), and the rotation of heads by it
  qkr    RMS norm of queries and keys, their rotation, and the write of fresh keys and values into cache rows, in one pass
  xattn  attention of ragged sequences of queries to padded encoder states of another length

``run`` computes them in elementary torch operations in 32 bits; with ``own`` set it calls the framework.
"""

import math

import torch

own = False

DEV = "cuda"
BYTES = {"bf16": 2, "f32": 4}
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token through a wide up-projection: a weight-streaming product
        {"name": "q8_token", "op": "q8", "M": 1, "K": 1536, "N": 8960},
        # QKV of a tenth of 32760 tokens
        {"name": "q8_qkv", "op": "q8", "M": 3276, "K": 1536, "N": 4608},
        # MLP down-projection with every token active
        {"name": "q8_down", "op": "q8", "M": 32760, "K": 8960, "N": 1536},
        # the table of a long text context, far positions, frequencies scaled by parts
        {"name": "rope_table_long", "op": "table", "P": 131072, "axes": 1, "rot": 128, "scaling": "parts", "far": 1000000},
        # a few rows, a part of the head, 32-bit rows
        {"name": "rope_few", "op": "rope", "n": 33, "H": 24, "d": 64, "rot": 32, "layout": "interleaved", "type": "f32"},
        # all queries of a 32760-token latent
        {"name": "rope_rows", "op": "rope", "n": 32760, "H": 12, "d": 128, "rot": 128, "layout": "half", "type": "bf16"},
        # half the tokens of a tiny latent
        {"name": "qkr_tiny", "op": "qkr", "N": 256, "n": 128, "H": 2, "d": 64, "rot": 64, "layout": "half", "norm": "head"},
        # 40 percent of 32760 video tokens, norm over the whole row
        {"name": "qkr_rows", "op": "qkr", "N": 32760, "n": 13104, "H": 12, "d": 128, "rot": 128, "layout": "interleaved", "norm": "row"},
        # a quarter of 75600 tokens of a wide model, norm of each head
        {"name": "qkr_wide", "op": "qkr", "N": 75600, "n": 18900, "H": 40, "d": 128, "rot": 128, "layout": "half", "norm": "head"},
        # one query per sequence, one sequence without keys
        {"name": "xattn_tokens", "op": "xattn", "B": 16, "n": 16, "H": 12, "Hk": 12, "d": 128, "S": 512, "mask": "len"},
        # a guided pair of latents and their padded prompts
        {"name": "xattn_text", "op": "xattn", "B": 2, "n": 26207, "H": 12, "Hk": 12, "d": 128, "S": 512, "mask": "len"},
        # long encoder states with holes, shared key heads
        {"name": "xattn_long", "op": "xattn", "B": 3, "n": 8190, "H": 12, "Hk": 4, "d": 128, "S": 4096, "mask": "holes"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["q8", "q8", "table", "rope", "qkr", "qkr", "xattn", "xattn"])
    d = rng.choice([64, 128])
    if op == "q8":
        while True:
            c = {"op": op, "M": _log(rng, 1, 32760), "K": _log(rng, 48, 8960), "N": _log(rng, 24, 8960)}
            if c["M"] * c["K"] * c["N"] <= 32760 * 8960 * 1536:
                return c
    if op == "table":
        axes = rng.choice([1, 2, 3])
        return {"op": op, "P": _log(rng, 1, 131072), "axes": axes, "rot": 16 * rng.randint(1, 8),
                "scaling": rng.choice(["none", "linear", "base", "parts"]), "far": _log(rng, 64, 1000000)}
    layout = rng.choice(["interleaved", "half"])
    rot = 16 * rng.randint(1, d // 16)
    if op == "rope":
        return {"op": op, "n": _log(rng, 1, 32760), "H": 128 // d * rng.randint(1, 12), "d": d, "rot": rot, "layout": layout,
                "type": rng.choice(["bf16", "f32"])}
    if op == "qkr":
        N = _log(rng, 64, 75600)
        return {"op": op, "N": N, "n": _log(rng, 1, max(1, N // 4)), "H": 128 // d * rng.randint(1, 40), "d": d, "rot": rot,
                "layout": layout, "norm": rng.choice(["none", "head", "row"])}
    B, S = _log(rng, 1, 24), _log(rng, 1, 4096)
    H = 128 // d * rng.choice([1, 2, 3, 4, 6, 8, 12])
    n = _log(rng, B, max(B, min(26207, 26207 * 512 * 12 // (S * H))))
    return {"op": op, "B": B, "n": n, "H": H, "Hk": rng.choice([h for h in (1, 2, 4, H // 2, H) if h and H % h == 0]), "d": d, "S": S,
            "mask": rng.choice(["len", "holes"])}


# ---------------------------------------------------------------- inputs

AXES = {1: (1.0,), 2: (0.5, 0.5), 3: (0.34, 0.33, 0.33)}


def _dims(rot, axes):
    """`rot` rotated places over the axes, an even number for each."""
    per = [max(2, int(rot * f) // 2 * 2) for f in AXES[axes]]
    per[0] += rot - sum(per)
    return per


def _starts(c):
    """Where each sequence's queries begin: about equal parts, one shifted into the other."""
    n, B = c["n"], c["B"]
    cuts = [n * b // B for b in range(B + 1)]
    return [x if b in (0, B) or B > n // 4 else min(n, x + (n // B) // 8) for b, x in enumerate(cuts)]


def _kv_lens(c):
    """Key counts from the whole padded length down to half of it; with four sequences or more the second has none."""
    B, S = c["B"], c["S"]
    lens = [max(1, S - b * S // (2 * B)) for b in range(B)]
    return [0 if B >= 4 and b == 1 else x for b, x in enumerate(lens)]


def _inv_freq(c, dims):
    """The frequencies of one axis in 64 bits; also the amplitude."""
    base, factor, orig, fast, slow = 10000.0, 8.0, 8192.0, 32.0, 1.0
    i = torch.arange(dims // 2, dtype=torch.float64, device=DEV)
    if c["scaling"] == "base" and dims > 2:
        base = base * factor ** (dims / (dims - 2))
    inv = base ** (-2.0 * i / dims)
    if c["scaling"] == "linear":
        inv = inv / factor
    if c["scaling"] == "parts":
        turns = orig * inv / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        inv = inv / factor * (1 - keep) + inv * keep
    return inv, (0.1 * math.log(factor) + 1.0 if c["scaling"] == "parts" else 1.0)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c, op = case, case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    if op == "q8":
        M, K, N = c["M"], c["K"], c["N"]
        a = (normal(M, K) * torch.exp(0.5 * normal(1, K))).to(torch.bfloat16)  # normalised rows, some channels larger
        w = normal(N, K) / math.sqrt(K)
        ws = w.abs().amax(1) / 127.0
        ld = (K + 15) // 16 * 16
        wq = torch.zeros(N, ld, dtype=torch.int8, device=DEV)
        wq[:, :K] = torch.round(w / ws[:, None]).to(torch.int8)
        return {"c": c, "a": a, "wq": wq, "ws": ws, "aq": torch.zeros(M, ld, dtype=torch.int8, device=DEV),
                "as": torch.empty(M, device=DEV), "out": torch.empty(M, N, dtype=torch.bfloat16, device=DEV)}
    if op == "table":
        pos = torch.randint(0, c["far"], (c["P"], c["axes"]), generator=g, device=DEV, dtype=torch.int32)
        return {"c": c, "pos": pos, "table": torch.empty(c["P"], c["rot"] // 2, 2, device=DEV)}
    if op == "rope":
        x = normal(c["n"], c["H"] * c["d"]).to(TYPE[c["type"]])
        table = _random_table(g, c["n"], c["rot"])
        return {"c": c, "x": x, "table": table, "y": torch.empty_like(x)}
    if op == "qkr":
        N, n, D = c["N"], c["n"], c["H"] * c["d"]
        qkv = normal(n, 3 * D).to(torch.bfloat16)
        idx = torch.sort(torch.randperm(N, generator=g, device=DEV)[:n]).values.to(torch.int32)
        width = D if c["norm"] == "row" else c["d"]
        return {"c": c, "qkv": qkv, "idx": idx, "w_q": 1 + 0.1 * normal(width), "w_k": 1 + 0.1 * normal(width),
                "table": _random_table(g, N, c["rot"]), "k_cache": normal(N, D).to(torch.bfloat16),
                "v_cache": normal(N, D).to(torch.bfloat16), "q": torch.empty(n, D, dtype=torch.bfloat16, device=DEV)}
    B, S, n, D = c["B"], c["S"], c["n"], c["H"] * c["d"]
    q = (2 * normal(n, D)).to(torch.bfloat16)
    k, v = normal(B, S, c["Hk"] * c["d"]).to(torch.bfloat16), normal(B, S, c["Hk"] * c["d"]).to(torch.bfloat16)
    starts = _starts(c)
    s = {"c": c, "q": q, "k": k, "v": v, "start": torch.tensor(starts, dtype=torch.int32, device=DEV),
         "longest": max(b - a for a, b in zip(starts, starts[1:])), "o": torch.empty_like(q),
         "len": torch.tensor(_kv_lens(c), dtype=torch.int32, device=DEV), "mask": None}
    if c["mask"] == "holes":
        s["mask"] = (torch.rand(B, S, generator=g, device=DEV) > 0.1).to(torch.uint8)
    return s


def _random_table(g, rows, rot):
    """Cosines and sines of angles as a table call leaves them."""
    a = torch.rand(rows, rot // 2, generator=g, device=DEV) * (2 * math.pi)
    return torch.stack([torch.cos(a), torch.sin(a)], dim=-1)


# ---------------------------------------------------------------- one pass

def run(state):
    return _OWN[state["c"]["op"]](state) if own else _PLAIN[state["c"]["op"]](state)


def _q8(s):
    K = s["c"]["K"]
    a = s["a"].float()
    amax = a.abs().amax(1, keepdim=True)
    aq = torch.round(a * (torch.full_like(amax, 127.0) / amax))
    acc = aq @ s["wq"][:, :K].float().t()
    return (acc * (amax / 127.0) * s["ws"]).to(torch.bfloat16)


def _table(s):
    c = s["c"]
    inv = [_inv_freq(c, r) for r in _dims(c["rot"], c["axes"])]
    a = torch.cat([s["pos"][:, x].double()[:, None] * f for x, (f, _) in enumerate(inv)], dim=1)
    return (torch.stack([torch.cos(a), torch.sin(a)], dim=-1) * inv[0][1]).float()


def _rotate(x, table, layout):
    """x [n, H, d] in 32 bits, its first places turned by the rows of the table."""
    half = table.shape[1]
    cos, sin = table[:, None, :, 0], table[:, None, :, 1]
    r, rest = x[..., : 2 * half], x[..., 2 * half:]
    if layout == "half":
        u, v = r[..., :half], r[..., half:]
        return torch.cat([u * cos - v * sin, v * cos + u * sin, rest], dim=-1)
    u, v = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([u * cos - v * sin, v * cos + u * sin], dim=-1).flatten(-2), rest], dim=-1)


def _rope(s):
    c, x = s["c"], s["x"]
    return _rotate(x.float().view(c["n"], c["H"], c["d"]), s["table"], c["layout"]).reshape(x.shape).to(x.dtype)


def _normed(x, w, norm):
    if norm == "none":
        return x
    flat = x.flatten(1) if norm == "row" else x
    return (flat * torch.rsqrt(flat.square().mean(-1, keepdim=True) + 1e-6) * w).view(x.shape)


def _qkr(s):
    c = s["c"]
    n, H, d = c["n"], c["H"], c["d"]
    D, rows = H * d, s["idx"].long()
    table = s["table"][rows]
    q, k, v = (s["qkv"][:, i * D:(i + 1) * D] for i in range(3))
    q = _rotate(_normed(q.float().view(n, H, d), s["w_q"], c["norm"]), table, c["layout"]).reshape(n, D)
    k = _rotate(_normed(k.float().view(n, H, d), s["w_k"], c["norm"]), table, c["layout"]).reshape(n, D)
    s["k_cache"][rows] = k.to(torch.bfloat16)
    s["v_cache"][rows] = v
    return q.to(torch.bfloat16), s["k_cache"], s["v_cache"]


def _xattn(s):
    c = s["c"]
    B, S, H, Hk, d = c["B"], c["S"], c["H"], c["Hk"], c["d"]
    row = torch.arange(c["n"], device=DEV)
    seq = torch.searchsorted(s["start"], row, right=True, out_int32=True).long() - 1
    at = row - s["start"][seq]
    q = torch.zeros(B, s["longest"], H, d, device=DEV)
    q[seq, at] = s["q"].float().view(c["n"], H, d)
    k = s["k"].float().view(B, S, Hk, d).repeat_interleave(H // Hk, dim=2)
    v = s["v"].float().view(B, S, Hk, d).repeat_interleave(H // Hk, dim=2)
    seen = torch.arange(S, device=DEV)[None, :] < s["len"][:, None]
    if s["mask"] is not None:
        seen = seen & (s["mask"] != 0)
    score = torch.matmul(q.permute(0, 2, 1, 3), k.permute(0, 2, 3, 1)) / math.sqrt(d)
    score.masked_fill_(~seen[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total == 0, torch.ones_like(total), total)
    return o.permute(0, 2, 1, 3)[seq, at].reshape(c["n"], H * d).to(torch.bfloat16)


_PLAIN = {"q8": _q8, "table": _table, "rope": _rope, "qkr": _qkr, "xattn": _xattn}


# ---------------------------------------------------------------- the framework's calls

_contexts = {}


def _ctx(N, H, d):
    """The handle that a program keeps for its model's shape."""
    from token_sparse_denoising_layer_b200 import abi

    if (N, H, d) not in _contexts:
        _contexts[N, H, d] = abi.hsa_create(N=N, D=H * d, H=H, F=64, L=0, T=1, budgets=[1], counts=[N])
    return abi, _contexts[N, H, d]


def _own_q8(s):
    c = s["c"]
    abi, ctx = _ctx(1, 1, 128)
    abi.hsa_quant_rows(ctx, s["a"], c["M"], c["K"], s["aq"], s["as"])
    abi.hsa_linear_quant(ctx, s["aq"], s["as"], c["M"], c["K"], s["wq"], s["ws"], c["N"], s["out"])
    return s["out"]


def _own_table(s):
    c = s["c"]
    abi, ctx = _ctx(1, 1, 128)
    cfg = abi.rope_cfg(_dims(c["rot"], c["axes"]), base=10000.0, scaling=c["scaling"], factor=8.0, orig_len=8192.0, fast=32.0,
                       slow=1.0, amp=0.1 * math.log(8.0) + 1.0 if c["scaling"] == "parts" else 1.0)
    abi.hsa_rope_table(ctx, cfg, s["pos"], c["P"], s["table"])
    return s["table"]


def _own_rope(s):
    c = s["c"]
    abi, ctx = _ctx(1, c["H"], c["d"])
    abi.hsa_rope(ctx, s["x"], c["n"], c["H"], s["table"], c["n"], c["rot"], s["y"], layout=c["layout"])
    return s["y"]


def _own_qkr(s):
    c = s["c"]
    D = c["H"] * c["d"]
    abi, ctx = _ctx(c["N"], c["H"], c["d"])
    how = abi.qk_rope(norm=c["norm"], w_q=s["w_q"], w_k=s["w_k"], eps=1e-6, table=s["table"], P=c["N"], rot=c["rot"], layout=c["layout"])
    qkv = s["qkv"]
    abi.hsa_qk_norm_rope(ctx, how, s["idx"], c["n"], s["q"], s["k_cache"], s["v_cache"], q_in=qkv[:, :D], k_in=qkv[:, D:2 * D],
                         v_in=qkv[:, 2 * D:])
    return s["q"], s["k_cache"], s["v_cache"]


def _own_xattn(s):
    c = s["c"]
    abi, ctx = _ctx(1, c["H"], c["d"])
    abi.hsa_cross_attention(ctx, s["q"], s["start"], c["n"], c["B"], s["k"], s["v"], c["S"], s["o"], kv_len=s["len"], kv_mask=s["mask"],
                            kv_heads=c["Hk"])
    return s["o"]


_OWN = {"q8": _own_q8, "table": _own_table, "rope": _own_rope, "qkr": _own_qkr, "xattn": _own_xattn}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    if op == "q8":
        M, K, N = c["M"], c["K"], c["N"]
        return {"bytes": 2 * M * K + N * K + 4 * N + 2 * M * N, "flops": 2 * M * K * N}
    if op == "table":
        return {"bytes": 4 * c["P"] * c["axes"] + 4 * c["P"] * c["rot"], "flops": c["P"] * c["rot"]}
    if op == "rope":
        b = BYTES[c["type"]]
        return {"bytes": 2 * b * c["n"] * c["H"] * c["d"] + 4 * c["n"] * c["rot"], "flops": 3 * c["n"] * c["H"] * c["rot"]}
    if op == "qkr":
        n, D = c["n"], c["H"] * c["d"]
        return {"bytes": 12 * n * D + 4 * n + 4 * n * c["rot"], "flops": 2 * n * (4 * D + 3 * c["H"] * c["rot"])}
    starts, lens = _starts(c), _kv_lens(c)
    pairs = sum((b - a) * x for a, b, x in zip(starts, starts[1:], lens))
    return {"bytes": 4 * c["n"] * c["H"] * c["d"] + 4 * sum(lens) * c["Hk"] * c["d"] + (sum(lens) if c["mask"] == "holes" else 0),
            "flops": 4 * pairs * c["H"] * c["d"]}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s, c = prepare(case, seed), case
    op = c["op"]
    if op == "q8":
        a = s["a"].double()
        scale = a.abs().max(dim=1).values.unsqueeze(1) / 127.0
        whole = torch.round(a / scale)
        return torch.mm(whole, s["wq"][:, :c["K"]].double().t()) * scale * s["ws"].double().unsqueeze(0)
    if op == "table":
        cols, amp = [], 1.0
        for x, dims in enumerate(_dims(c["rot"], c["axes"])):
            for i in range(dims // 2):
                b = 10000.0 * 8.0 ** (dims / (dims - 2)) if c["scaling"] == "base" and dims > 2 else 10000.0
                f = math.pow(b, -2.0 * i / dims)
                if c["scaling"] == "linear":
                    f /= 8.0
                if c["scaling"] == "parts":
                    amp = 1.0 + 0.1 * math.log(8.0)
                    share = min(1.0, max(0.0, (8192.0 * f / (2 * math.pi) - 1.0) / 31.0))
                    f = share * f + (1.0 - share) * f / 8.0
                ang = s["pos"][:, x].double() * f
                cols.append(torch.stack((ang.cos() * amp, ang.sin() * amp), dim=1))
        return torch.stack(cols, dim=1)
    if op == "rope":
        z = s["x"].double().reshape(c["n"], c["H"], c["d"])
        return _turn64(z, s["table"].double(), c["layout"]).reshape(c["n"], -1)
    if op == "qkr":
        n, H, d = c["n"], c["H"], c["d"]
        D, at = H * d, s["idx"].long()
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        out = []
        for part, w in ((0, s["w_q"]), (1, s["w_k"])):
            z = s["qkv"][:, part * D:(part + 1) * D].double()
            if c["norm"] == "row":
                z = z / torch.sqrt((z * z).sum(1, keepdim=True) / D + 1e-6) * w.double()
            z = z.reshape(n, H, d)
            if c["norm"] == "head":
                z = z / torch.sqrt((z * z).sum(2, keepdim=True) / d + 1e-6) * w.double()
            out.append(_turn64(z, s["table"].double().index_select(0, at), c["layout"]).reshape(n, D))
        kc.index_copy_(0, at, out[1])
        vc.index_copy_(0, at, s["qkv"][:, 2 * D:].double())
        return out[0], kc, vc
    starts, lens = _starts(c), _kv_lens(c)
    H, Hk, d = c["H"], c["Hk"], c["d"]
    o = torch.zeros(c["n"], H, d, dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        keys = torch.arange(lens[b], device=DEV)
        if s["mask"] is not None:
            keys = keys[s["mask"][b, :lens[b]] != 0]
        if starts[b] == starts[b + 1] or keys.numel() == 0:
            continue
        for h in range(H):
            kv = slice(h // (H // Hk) * d, (h // (H // Hk) + 1) * d)
            k, v = s["k"][b, keys, kv].double(), s["v"][b, keys, kv].double()
            q = s["q"][starts[b]:starts[b + 1], h * d:(h + 1) * d].double()
            o[starts[b]:starts[b + 1], h] = torch.softmax(q @ k.t() * d ** -0.5, dim=1) @ v
    return o.reshape(c["n"], H * d)


def _turn64(z, table, layout):
    """The rotation as a product of complex numbers."""
    half = table.shape[1]
    turn = torch.complex(table[..., 0], table[..., 1]).unsqueeze(1)
    y = z.clone()
    if layout == "half":
        w = torch.complex(z[..., :half], z[..., half:2 * half]) * turn
        y[..., :half], y[..., half:2 * half] = w.real, w.imag
    else:
        w = torch.complex(z[..., 0:2 * half:2].contiguous(), z[..., 1:2 * half:2].contiguous()) * turn
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = w.real, w.imag
    return y
