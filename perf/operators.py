"""The serving and training operators around the attention kernels, as measured cases.

qk_norm_rope      RMS norm of every query and key head and the rotation by position, in one pass
qk_norm_rope_bwd  its gradients
cache             the same for the new tokens of a serving step, with K and V written to a paged cache
decode            one new token per sequence against the paged cache
sinks_fwd         attention with a sliding window and a few first tokens that stay visible
sinks_bwd         its gradients

`own` selects who computes: the plain form below in elementary torch operations, or the framework.
"""
import math

import torch

own = False

DEV = "cuda"
PHI = 0.6180339887498949


def listed():
    return [
        # A training batch at the library's headline shape, before attention.
        dict(name="norm_rope train", op="qk_norm_rope", B=2, S=8192, Hq=16, Hkv=16, D=128, R=128,
             interleaved=False),
        # The gradients of a short odd batch: two query heads per key head, part of the head rotated in pairs.
        dict(name="norm_rope bwd odd", op="qk_norm_rope_bwd", B=3, S=333, Hq=6, Hkv=2, D=64, R=48,
             interleaved=True),
        # The gradients of a long grouped-head training sequence.
        dict(name="norm_rope bwd long", op="qk_norm_rope_bwd", B=1, S=16384, Hq=32, Hkv=8, D=128, R=128,
             interleaved=False),
        # One new token of one stream: latency.
        dict(name="cache write 1 token", op="cache", T=1, Hq=32, Hkv=8, D=128, R=128, interleaved=False,
             kv="bf16", page=16, pages=64),
        # A prefill chunk into an 8-bit cache.
        dict(name="cache write chunk fp8", op="cache", T=4099, Hq=32, Hkv=8, D=128, R=64, interleaved=False,
             kv="fp8", page=64, pages=128),
        # One user's stream, about a thousand tokens in: latency.
        dict(name="decode 1 x 1000", op="decode", B=1, L=1000, ragged=False, Hq=32, Hkv=8, D=128, kv="bf16",
             page=16, window=-1, sinks=0),
        # A serving batch of unequal lengths.
        dict(name="decode 64 ragged", op="decode", B=64, L=8192, ragged=True, Hq=32, Hkv=8, D=128, kv="bf16",
             page=16, window=-1, sinks=0),
        # Long contexts in an 8-bit cache.
        dict(name="decode 8 x 131072 fp8", op="decode", B=8, L=131072, ragged=False, Hq=32, Hkv=8, D=128, kv="fp8",
             page=64, window=-1, sinks=0),
        # Endless streams: a window of 4096 keys and four first tokens, as many key heads as query heads.
        dict(name="decode window sinks", op="decode", B=33, L=16384, ragged=True, Hq=16, Hkv=16, D=128,
             kv="bf16", page=32, window=4095, sinks=4),
        # The headline training shape under a 1024-key window with four sinks.
        dict(name="sinks fwd train", op="sinks_fwd", B=2, Sq=8192, Sk=8192, Hq=16, Hkv=16, D=128, window=1023,
             sinks=4),
        # The next chunk of a prompt against what is there already, odd sizes, small heads.
        dict(name="sinks fwd chunk", op="sinks_fwd", B=1, Sq=777, Sk=2345, Hq=8, Hkv=2, D=64, window=500,
             sinks=130),
        # The backward's training shape under the same window.
        dict(name="sinks bwd train", op="sinks_bwd", B=2, Sq=4096, Sk=4096, Hq=16, Hkv=16, D=128, window=1023,
             sinks=4),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


HEADS = [(16, 16), (32, 8), (24, 24), (8, 1), (6, 2), (2, 2), (40, 2), (8, 2), (32, 1)]


def draw(rng):
    op = rng.choice(["qk_norm_rope", "qk_norm_rope_bwd", "cache", "decode", "decode", "sinks_fwd", "sinks_bwd"])
    Hq, Hkv = rng.choice(HEADS)
    D = rng.choice([64, 128, 128])
    if op in ("qk_norm_rope", "qk_norm_rope_bwd"):
        B = rng.randint(1, 4)
        S = _log_int(rng, 1, max(1, 4_000_000 // (B * (Hq + Hkv) * D // 16)))
        return dict(op=op, B=B, S=S, Hq=Hq, Hkv=Hkv, D=D, R=rng.choice([D, D, D // 2, 16]),
                    interleaved=rng.random() < 0.4)
    if op == "cache":
        page = rng.choice([16, 32, 48, 64, 128])
        T = _log_int(rng, 1, 6000)
        return dict(op=op, T=T, Hq=Hq, Hkv=Hkv, D=D, R=rng.choice([D, D // 2, 16]), interleaved=rng.random() < 0.4,
                    kv=rng.choice(["bf16", "fp8"]), page=page, pages=T // page + rng.randint(2, 40))
    if op == "decode":
        kv = rng.choice(["bf16", "fp8"])
        L = _log_int(rng, 1, 131072)
        most = 600_000_000 // (L * Hkv * D)
        B = _log_int(rng, 1, max(1, min(200, most)))
        window = rng.choice([-1, -1, _log_int(rng, 1, 8192) - 1])
        return dict(op=op, B=B, L=L, ragged=rng.random() < 0.6, Hq=Hq, Hkv=Hkv, D=D, kv=kv,
                    page=rng.choice([16, 32, 48, 64, 128]), window=window,
                    sinks=0 if window < 0 else rng.choice([0, 1, 4, 17, 128]))
    B = rng.randint(1, 3)
    # The plain form holds every score of every head: up to 2^29 of them here.
    # (A backward over one key alone has gradients of zero, which rounding hides: it starts at 16.)
    Sk = _log_int(rng, 16 if op == "sinks_bwd" else 1, 6000 if Hq * B <= 16 else 3500)
    Sq = Sk if rng.random() < 0.6 else _log_int(rng, 1, Sk)
    if rng.random() < 0.15:  # more queries than keys: the first rows see none
        Sq = Sk + rng.randint(1, 200)
    return dict(op=op, B=B, Sq=Sq, Sk=Sk, Hq=Hq, Hkv=Hkv, D=D, window=_log_int(rng, 1, 2048) - 1,
                sinks=rng.choice([1, 4, 17, 128, 200]))


# ------------------------------------------------------------------ inputs

def _lens(case):
    """Lengths of a batch, the new token counted: all L, or spread over (0, L] by the case alone."""
    if not case["ragged"]:
        return [case["L"]] * case["B"]
    return [1 + int((case["L"] - 1) * (((i + 1) * PHI) % 1.0)) for i in range(case["B"])]


def _table(n, R, theta=10000.0):
    inv = theta ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R)
    ang = torch.arange(n, dtype=torch.float64, device=DEV)[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def _randn(g, *shape, dtype=torch.bfloat16, std=1.0):
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16 if dtype != torch.float32 else dtype)
    return x * std if std != 1.0 else x


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    c, s = case, dict(case=case)
    if c["op"] in ("qk_norm_rope", "qk_norm_rope_bwd"):
        # Q and K are views of one projection's output [B, S, (Hq + 2 Hkv) D].
        qkv = _randn(g, c["B"], c["S"], (c["Hq"] + 2 * c["Hkv"]) * c["D"])
        s["q"] = qkv[..., :c["Hq"] * c["D"]].unflatten(-1, (c["Hq"], c["D"]))
        s["k"] = qkv[..., c["Hq"] * c["D"]:(c["Hq"] + c["Hkv"]) * c["D"]].unflatten(-1, (c["Hkv"], c["D"]))
        s["qw"], s["kw"] = (1 + _randn(g, c["D"], std=0.1) for _ in range(2))
        s["cos"], s["sin"] = _table(c["S"], c["R"])
        s["pos"] = torch.arange(c["S"], dtype=torch.int32, device=DEV).repeat(c["B"], 1)
        if c["op"].endswith("bwd"):
            s["dq"] = _randn(g, c["B"], c["S"], c["Hq"], c["D"], dtype=torch.float32)
            s["dk"] = _randn(g, c["B"], c["S"], c["Hkv"], c["D"])
    elif c["op"] == "cache":
        qkv = _randn(g, c["T"], (c["Hq"] + 2 * c["Hkv"]) * c["D"])
        s["q"], s["k"], s["v"] = (x.unflatten(-1, (-1, c["D"])) for x in qkv.split(
            [c["Hq"] * c["D"], c["Hkv"] * c["D"], c["Hkv"] * c["D"]], -1))
        s["qw"], s["kw"] = (1 + _randn(g, c["D"], std=0.1) for _ in range(2))
        s["cos"], s["sin"] = _table(8192, c["R"])
        s["pos"] = (torch.arange(c["T"], dtype=torch.int32, device=DEV) + 17) % 8192
        n = c["pages"] * c["page"]
        s["slots"] = torch.randperm(n, generator=g, device=DEV)[:c["T"]].to(torch.int32)
        s["descale"] = 1.0 / 64 if c["kv"] == "fp8" else 1.0
        for name in ("kc", "vc"):
            s[name] = _cache(g, c["kv"], c["pages"], c["page"], c["Hkv"], c["D"])
    elif c["op"] == "decode":
        lens = _lens(c)
        width = -(-max(lens) // c["page"])
        need = [-(-n // c["page"]) for n in lens]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = torch.zeros(c["B"], width, dtype=torch.int32, device=DEV)
        row = torch.repeat_interleave(torch.arange(c["B"]), torch.tensor(need))
        first = torch.tensor([0] + need[:-1]).cumsum(0)
        col = torch.arange(sum(need)) - first[row]
        table[row.to(DEV), col.to(DEV)] = order[:sum(need)]
        s["table"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["q"] = _randn(g, c["B"], c["Hq"], c["D"])
        s["descale"] = 1.0 / 64 if c["kv"] == "fp8" else 1.0
        for name in ("kc", "vc"):
            s[name] = _cache(g, c["kv"], pages, c["page"], c["Hkv"], c["D"])
    else:
        s["q"] = _randn(g, c["B"], c["Sq"], c["Hq"], c["D"])
        s["k"], s["v"] = (_randn(g, c["B"], c["Sk"], c["Hkv"], c["D"]) for _ in range(2))
        if c["op"] == "sinks_bwd":
            s["dout"] = _randn(g, c["B"], c["Sq"], c["Hq"], c["D"])
            s["o"], s["lse"] = _attention(c, s["q"], s["k"], s["v"])
    return s


def _cache(g, kv, pages, page, Hkv, D):
    x = _randn(g, pages, page, Hkv, D)
    return (x * 64).to(torch.float8_e4m3fn) if kv == "fp8" else x


# -------------------------------------------------------------- plain forms

def _norm(x, w, eps=1e-6):
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    return x * r, r, w.float()


def _halves(x, R, interleaved):
    """The two members of every rotated pair, and what is not rotated."""
    rot = x[..., :R]
    if interleaved:
        return rot[..., 0::2], rot[..., 1::2], x[..., R:]
    return rot[..., :R // 2], rot[..., R // 2:], x[..., R:]


def _join(a, b, rest, interleaved):
    rot = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((rot, rest), -1)


def _rotate(x, cos, sin, R, interleaved):
    a, b, rest = _halves(x, R, interleaved)
    return _join(a * cos - b * sin, b * cos + a * sin, rest, interleaved)


def _angles(s):
    pos = s["pos"].long()
    return s["cos"][pos].unsqueeze(-2), s["sin"][pos].unsqueeze(-2)


def _norm_rope(s, x, w):
    c = s["case"]
    xr, _, wf = _norm(x, w)
    return _rotate(xr * wf, *_angles(s), c["R"], c["interleaved"])


def _norm_rope_grad(s, dy, x, w):
    c = s["case"]
    xr, r, wf = _norm(x, w)
    cos, sin = _angles(s)
    g = _rotate(dy.float(), cos, -sin, c["R"], c["interleaved"])
    h = g * wf
    dx = r * (h - xr * (h * xr).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (g * xr).sum((0, 1, 2))


def _codes(x, kv, descale):
    return x.to(torch.bfloat16) if kv == "bf16" else (x / descale).clamp(-448, 448).to(torch.float8_e4m3fn)


def _put(cache, slots, rows):
    flat = cache.view(torch.uint8 if cache.dtype == torch.float8_e4m3fn else cache.dtype).flatten(0, 1)
    flat[slots.long()] = rows.view(flat.dtype)


def _visible(c):
    """[Sq, Sk] of the keys that a query may see."""
    i = torch.arange(c["Sq"], device=DEV)[:, None] + (c["Sk"] - c["Sq"])
    j = torch.arange(c["Sk"], device=DEV)[None, :]
    return (j <= i) & ((j >= i - c["window"]) | (j < c["sinks"]))


def _heads(x, Hq):
    """[B, S, H, D] as fp32 [B, Hq, S, D], key heads repeated for their group."""
    x = x.float().transpose(1, 2)
    return x.repeat_interleave(Hq // x.shape[1], 1)


def _attention(c, q, k, v):
    s = _heads(q, c["Hq"]) @ _heads(k, c["Hq"]).transpose(-1, -2) * c["D"] ** -0.5
    s = s.masked_fill_(~_visible(c), -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min(-1e30)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p @ _heads(v, c["Hq"])) / l.clamp_min(1e-30)
    return o.transpose(1, 2).contiguous().to(torch.bfloat16), (m + l.log()).squeeze(-1)


def _attention_grad(s):
    c = s["case"]
    q, k, v, dout = (_heads(s[n], c["Hq"]) for n in ("q", "k", "v", "dout"))
    scale = c["D"] ** -0.5
    lse = s["lse"].unsqueeze(-1)
    p = (q @ k.transpose(-1, -2)).mul_(scale).sub_(lse.nan_to_num(neginf=0.0)).exp_()
    p = p.masked_fill_(~_visible(c), 0.0)
    delta = (dout * _heads(s["o"], c["Hq"])).sum(-1, keepdim=True)
    dv = p.transpose(-1, -2) @ dout
    ds = (dout @ v.transpose(-1, -2)).sub_(delta).mul_(p)
    dq = ds @ k * scale
    dk = ds.transpose(-1, -2) @ q * scale
    G = c["Hq"] // c["Hkv"]
    dk, dv = (x.unflatten(1, (c["Hkv"], G)).sum(2) for x in (dk, dv))
    return tuple(x.transpose(1, 2).contiguous().to(torch.bfloat16) for x in (dq, dk, dv))


def _decode(s):
    c = s["case"]
    n = s["table"].shape[1] * c["page"]
    j = torch.arange(n, device=DEV)[None, :]
    end = s["lens"][:, None]
    see = j < end
    if c["window"] >= 0:
        see &= (j >= end - 1 - c["window"]) | (j < c["sinks"])
    G = c["Hq"] // c["Hkv"]
    q = s["q"].float().unflatten(1, (c["Hkv"], G)) * c["D"] ** -0.5
    k = s["kc"][s["table"].long()].flatten(1, 2).float().mul_(s["descale"])  # [B, n, Hkv, D]
    x = q @ k.permute(0, 2, 3, 1)
    del k
    x = x.masked_fill_(~see[:, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    v = s["vc"][s["table"].long()].flatten(1, 2).float().mul_(s["descale"])
    o = (p @ v.transpose(1, 2)) / l
    return o.flatten(1, 2).to(torch.bfloat16), (m + l.log()).flatten(1)


def _plain(s):
    c = s["case"]
    if c["op"] == "qk_norm_rope":
        return tuple(_norm_rope(s, s[n], s[w]).to(torch.bfloat16) for n, w in (("q", "qw"), ("k", "kw")))
    if c["op"] == "qk_norm_rope_bwd":
        dq, dqw = _norm_rope_grad(s, s["dq"], s["q"], s["qw"])
        dk, dkw = _norm_rope_grad(s, s["dk"], s["k"], s["kw"])
        return dq, dk, dqw, dkw
    if c["op"] == "cache":
        q = _norm_rope(s, s["q"], s["qw"]).to(torch.bfloat16)
        _put(s["kc"], s["slots"], _codes(_norm_rope(s, s["k"], s["kw"]), c["kv"], s["descale"]))
        _put(s["vc"], s["slots"], _codes(s["v"].float(), c["kv"], s["descale"]))
        return q, s["kc"], s["vc"]
    if c["op"] == "decode":
        return _decode(s)
    if c["op"] == "sinks_fwd":
        return _attention(c, s["q"], s["k"], s["v"])
    return _attention_grad(s)


def run(s):
    if not own:
        return _plain(s)
    from tiled_attention_blackwell_b200 import attn
    c = s["case"]
    if c["op"] == "qk_norm_rope":
        return attn.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["cos"], s["sin"], s["pos"],
                                 interleaved=c["interleaved"])
    if c["op"] == "qk_norm_rope_bwd":
        return attn.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["qw"], s["kw"], s["cos"], s["sin"],
                                          s["pos"], interleaved=c["interleaved"])
    if c["op"] == "cache":
        q = attn.qk_norm_rope_cache(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["cos"], s["sin"], s["pos"],
                                    s["slots"], s["kc"], s["vc"], k_descale=s["descale"], v_descale=s["descale"],
                                    interleaved=c["interleaved"])
        return q, s["kc"], s["vc"]
    if c["op"] == "decode":
        return attn.decode_paged(s["q"], s["kc"], s["vc"], s["table"], s["lens"], k_descale=s["descale"],
                                 v_descale=s["descale"], sinks=c["sinks"],
                                 window=None if c["window"] < 0 else (c["window"], 0))
    if c["op"] == "sinks_fwd":
        return attn.attention(s["q"], s["k"], s["v"], causal=True, window=(c["window"], 0), sinks=c["sinks"])
    dq, dk, dv = attn.attention_backward(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dout"], causal=True,
                                         window=(c["window"], 0), sinks=c["sinks"])
    return dq.to(torch.bfloat16), dk, dv  # gradients of bf16 tensors, in their type


# --------------------------------------------------------------------- work

def _pairs(c):
    """(query, key) pairs that the mask leaves, of one head."""
    total = 0
    for i in range(c["Sq"]):
        d = i + c["Sk"] - c["Sq"]
        if d >= 0:
            lo = max(0, d - c["window"])
            total += d - lo + 1 + min(c["sinks"], lo)
    return total


def work(case):
    c = case
    if c["op"] in ("qk_norm_rope", "qk_norm_rope_bwd"):
        tokens = c["B"] * c["S"]
        q, k = tokens * c["Hq"] * c["D"], tokens * c["Hkv"] * c["D"]
        small = c["S"] * c["R"] * 4 + tokens * 4 + 4 * c["D"]
        if c["op"] == "qk_norm_rope":
            return {"bytes": 4 * (q + k) + small, "flops": 9 * (q + k)}
        return {"bytes": 8 * q + 6 * k + small + 8 * c["D"], "flops": 18 * (q + k)}
    if c["op"] == "cache":
        q, k = c["T"] * c["Hq"] * c["D"], c["T"] * c["Hkv"] * c["D"]
        out = 1 if c["kv"] == "fp8" else 2
        return {"bytes": 4 * q + 2 * k * (2 + out) + c["T"] * (c["R"] * 4 + 8) + 4 * c["D"], "flops": 9 * (q + k)}
    if c["op"] == "decode":
        keys = 0
        for n in _lens(c):
            lo = max(0, n - 1 - c["window"]) if c["window"] >= 0 else 0
            keys += n - lo + min(c["sinks"], lo)
        size = 1 if c["kv"] == "fp8" else 2
        io = c["B"] * c["Hq"] * (4 * c["D"] + 4)
        return {"bytes": 2 * keys * c["Hkv"] * c["D"] * size + io, "flops": 4 * keys * c["Hq"] * c["D"]}
    q, k = c["B"] * c["Sq"] * c["Hq"] * c["D"], c["B"] * c["Sk"] * c["Hkv"] * c["D"]
    rows = c["B"] * c["Sq"] * c["Hq"]
    if c["op"] == "sinks_fwd":
        return {"bytes": 4 * q + 4 * k + 4 * rows, "flops": 4 * c["B"] * c["Hq"] * c["D"] * _pairs(c)}
    return {"bytes": 8 * q + 8 * k + 4 * rows, "flops": 10 * c["B"] * c["Hq"] * c["D"] * _pairs(c)}


# -------------------------------------------------------- 64-bit definitions

def _exact_rotation(s):
    """Complex factors [tokens..., 1, R / 2] of the given table."""
    pos = s["pos"].long()
    return torch.complex(s["cos"].double(), s["sin"].double())[pos].unsqueeze(-2)


def _as_pairs(x, R, interleaved):
    a = x[..., :R].double()
    a = a.unflatten(-1, (R // 2, 2)) if interleaved else a.unflatten(-1, (2, R // 2)).transpose(-1, -2)
    return torch.view_as_complex(a.contiguous())


def _from_pairs(z, like, R, interleaved):
    y = like.double().clone()
    a = torch.view_as_real(z)
    y[..., :R] = (a if interleaved else a.transpose(-1, -2)).flatten(-2)
    return y


def _exact_norm_rope(s, x, w):
    c = s["case"]
    x = x.double()
    u = w.double() * x / (x.pow(2).sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt()
    return _from_pairs(_as_pairs(u, c["R"], c["interleaved"]) * _exact_rotation(s), u, c["R"], c["interleaved"])


def _exact_norm_rope_grad(s, dy, x, w):
    c = s["case"]
    dy, x, w = dy.double(), x.double(), w.double()
    g = _from_pairs(_as_pairs(dy, c["R"], c["interleaved"]) * _exact_rotation(s).conj(), dy, c["R"],
                    c["interleaved"])
    ms = x.pow(2).sum(-1, keepdim=True) / c["D"] + 1e-6
    dot = (w * g * x).sum(-1, keepdim=True)
    dx = w * g / ms.sqrt() - x * dot / (c["D"] * ms.pow(1.5))
    return dx, (g * x / ms.sqrt()).flatten(0, -2).sum(0)


def _exact_head(c, q, k, v):
    """Probabilities, output and LSE of one head: q [Sq, D], k, v [Sk, D]."""
    s = q.double() @ k.double().T / math.sqrt(c["D"])
    s[~_visible(c)] = -math.inf
    lse = torch.logsumexp(s, -1)
    p = torch.where(torch.isinf(s), 0.0, (s - lse[:, None]).exp())
    return p @ v.double(), lse


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "qk_norm_rope":
        return _exact_norm_rope(s, s["q"], s["qw"]), _exact_norm_rope(s, s["k"], s["kw"])
    if c["op"] == "qk_norm_rope_bwd":
        dq, dqw = _exact_norm_rope_grad(s, s["dq"], s["q"], s["qw"])
        dk, dkw = _exact_norm_rope_grad(s, s["dk"], s["k"], s["kw"])
        return dq, dk, dqw, dkw
    if c["op"] == "cache":
        at = s["slots"].long()
        out = [_exact_norm_rope(s, s["q"], s["qw"])]
        for cache, rows in ((s["kc"], _exact_norm_rope(s, s["k"], s["kw"])), (s["vc"], s["v"].double())):
            full = cache.double().flatten(0, 1)
            full[at] = (rows / s["descale"]).clamp(-448, 448) if c["kv"] == "fp8" else rows
            out.append(full.view(cache.shape))
        return tuple(out)
    G = c["Hq"] // c["Hkv"]
    if c["op"] == "decode":
        o = torch.zeros(c["B"], c["Hq"], c["D"], dtype=torch.float64, device=DEV)
        lse = torch.zeros(c["B"], c["Hq"], dtype=torch.float64, device=DEV)
        for b, n in enumerate(_lens(c)):
            lo = max(0, n - 1 - c["window"]) if c["window"] >= 0 else 0
            keys = torch.cat((torch.arange(min(c["sinks"], lo)), torch.arange(lo, n))).to(DEV)
            page = s["table"][b].long()[keys // c["page"]]
            kb, vb = (s[name][page, keys % c["page"]].double() * s["descale"] for name in ("kc", "vc"))
            for h in range(c["Hkv"]):
                hs = slice(h * G, h * G + G)
                x = s["q"][b, hs].double() @ kb[:, h].T / math.sqrt(c["D"])
                lse[b, hs] = torch.logsumexp(x, -1)
                o[b, hs] = torch.softmax(x, -1) @ vb[:, h]
        return o, lse
    if c["op"] == "sinks_fwd":
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.zeros(c["B"], c["Hq"], c["Sq"], dtype=torch.float64, device=DEV)
        for b in range(c["B"]):
            for h in range(c["Hq"]):
                o[b, :, h], lse[b, h] = _exact_head(c, s["q"][b, :, h], s["k"][b, :, h // G], s["v"][b, :, h // G])
        return o, lse
    dq = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    dk, dv = (torch.zeros(s["k"].shape, dtype=torch.float64, device=DEV) for _ in range(2))
    see = _visible(c)
    for b in range(c["B"]):
        for h in range(c["Hq"]):
            q, do, o = (s[n][b, :, h].double() for n in ("q", "dout", "o"))
            k, v = (s[n][b, :, h // G].double() for n in ("k", "v"))
            p = torch.where(see, (q @ k.T / math.sqrt(c["D"]) - s["lse"][b, h].double()[:, None]).exp(), 0.0)
            ds = p * (do @ v.T - (do * o).sum(-1, keepdim=True))
            dq[b, :, h] = ds @ k / math.sqrt(c["D"])
            dk[b, :, h // G] += ds.T @ q / math.sqrt(c["D"])
            dv[b, :, h // G] += p.T @ do
    return dq, dk, dv
