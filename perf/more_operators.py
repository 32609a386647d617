"""Rotary positions, the rotated cache append and the fused residual norms: what is timed, and their plain forms.

Three operators around the projections and the attention of a W4A4 transformer block, over the sizes they meet:
  * kq_rope              an optional norm of each head, then rotary positions with one to four axes;
  * kq_cache_write_rope  the same for the queries and keys of a fused projection, the keys and values going on to their
                         slots of the MXFP4 cache (read back here with kq_cache_read, as the values they stand for);
  * kq_residual_norm     x' = a x + gate * norm(y), then the next block's norm and modulation of x', in bf16, in MXFP4
                         (read back likewise) or as row statistics for the quantizer that follows.

`own = False` computes them with elementary torch operations; `own = True` calls the library.
"""
import math

import torch

own = False

DEV = "cuda:0"
EPS = 1e-6

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes by code; bit 3 is the sign
BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # between them; at a border the even code is taken


# ---------------------------------------------------------------- cases

def listed():
    return [
        # eight sequences' queries at one new token each, far into their contexts: all latency
        dict(name="rope_step", kind="rope", tokens=8, seqs=8, heads=32, dim=128, axes="128", halves=True, norm=True,
             far=900000),
        # image tokens of a guidance batch at the 1152-wide transformer: rows and columns, heads of 72, no norm
        dict(name="rope_image", kind="rope", tokens=8192, seqs=2, heads=16, dim=72, axes="36+36", halves=False,
             norm=False, far=0),
        # a video's queries: time, height and width, normalised heads of 128, an odd number of tokens
        dict(name="rope_video", kind="rope", tokens=32761, seqs=1, heads=16, dim=128, axes="16+56+56", halves=False,
             norm=True, far=0),
        # the decode step of eight sequences: queries, keys and values of a fused projection, grouped heads
        dict(name="append_step", kind="append", tokens=8, seqs=8, q_heads=32, kv_heads=8, dim=128, axes="128",
             halves=True, norm=True, far=900000, page=64, slots=4096, padded=1),
        # keys and values alone of an image at the 1152-wide transformer: heads of 72, whose blocks of 32 span two heads
        dict(name="append_image", kind="append", tokens=4095, seqs=1, q_heads=0, kv_heads=16, dim=72, axes="36+36",
             halves=False, norm=True, far=0, page=100, slots=8000, padded=31),
        # prompt chunks with rotation of a part of each head, as halves; heads of 96
        dict(name="append_partial", kind="append", tokens=6001, seqs=3, q_heads=20, kv_heads=10, dim=96, axes="64",
             halves=True, norm=False, far=20000, page=50, slots=16000, padded=0),
        # a long prompt: every head of a fused projection, an odd token count
        dict(name="append_prompt", kind="append", tokens=20481, seqs=1, q_heads=32, kv_heads=8, dim=128, axes="128",
             halves=True, norm=True, far=100000, page=64, slots=32768, padded=0),
        # the decode step of eight sequences: a gated residual with norms on both sides, quantised
        dict(name="norm_step", kind="norm", tokens=8, d=2240, samples=1, post="rms", gate=False, weights=True, pre="rms",
             modulate=False, scale=1.0, out="codes"),
        # the 1152-wide transformer's AdaLN between attention and MLP, a guidance batch, quantised for the next product
        dict(name="norm_adaln", kind="norm", tokens=8192, d=1152, samples=2, post="none", gate=True, weights=False,
             pre="layer", modulate=True, scale=1.0, out="codes"),
        # the residual stream of the 2240-wide transformer and the statistics that its quantizer reads
        dict(name="norm_stats", kind="norm", tokens=4097, d=2240, samples=1, post="none", gate=True, weights=False,
             pre="layer", modulate=False, scale=1.0, out="stats"),
        # norms before and after a block, gated and modulated, a scaled residual, bf16 for the next product
        dict(name="norm_sandwich", kind="norm", tokens=18432, d=2240, samples=4, post="rms", gate=True, weights=True,
             pre="rms", modulate=True, scale=0.5, out="rows"),
        # few and very wide rows: the wide MLP input
        dict(name="norm_wide", kind="norm", tokens=1009, d=12288, samples=1, post="layer", gate=False, weights=True,
             pre="layer", modulate=True, scale=1.0, out="codes"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("rope", "append", "append", "norm", "norm"))
    if kind == "norm":
        while True:
            tokens, d = _log(rng, 1, 18432), 32 * _log(rng, 2, 512)
            if tokens * d <= 18432 * 2240:
                break
        return dict(kind="norm", tokens=tokens, d=d, samples=rng.randint(1, min(4, tokens)),
                    post=rng.choice(("none", "rms", "layer")), gate=rng.random() < 0.6, weights=rng.random() < 0.5,
                    pre=rng.choice(("rms", "layer")), modulate=rng.random() < 0.6, scale=rng.choice((1.0, 1.0, 0.5)),
                    out=rng.choice(("codes", "codes", "rows", "stats")))
    dim = rng.choice((32, 40, 64, 72, 80, 96, 112, 128))
    n = rng.choice((1, 1, 2, 3))
    halves = rng.random() < 0.5
    turned = dim if rng.random() < 0.7 else dim // 16 * 8  # channels that turn
    first = turned - 2 * (turned // 2 // n) * (n - 1)
    axes = "+".join(str(v) for v in [first] + [2 * (turned // 2 // n)] * (n - 1))
    base = dict(kind=kind, dim=dim, axes=axes, halves=halves, norm=rng.random() < 0.6,
                far=_log(rng, 1, 1000000) if n == 1 else 0)
    if kind == "rope":
        heads = rng.choice((1, 3, 8, 16, 20, 32))
        while True:
            tokens = _log(rng, 1, 40000)
            if tokens * heads * dim <= 32761 * 2048:
                return dict(base, tokens=tokens, seqs=rng.randint(1, min(8, tokens)), heads=heads)
    kv_heads = rng.choice([h for h in (1, 2, 4, 5, 8, 12, 16, 20) if h * dim % 32 == 0])
    group = rng.choice((0, 1, 2, 4, 8))
    page = rng.choice((16, 50, 64, 128, 300))
    while True:
        tokens = _log(rng, 1, 40000)
        if tokens * kv_heads * (group + 2) * dim <= 20481 * 48 * 128:
            break
    return dict(base, tokens=tokens, seqs=rng.randint(1, min(8, tokens)), q_heads=group * kv_heads, kv_heads=kv_heads,
                page=page, slots=page * (-(-tokens // page) + rng.randint(1, 40)),
                padded=rng.choice((0, min(tokens - 1, 5))))


def work(case):
    t = case["tokens"]
    if case["kind"] == "norm":
        n = t * case["d"]
        out = {"codes": 17 / 32 * 2 + 2, "rows": 2, "stats": 0}[case["out"]]  # codes are read back as values
        vectors = 2 * case["weights"] + (case["gate"] + 2 * case["modulate"]) * case["samples"]
        return {"bytes": n * (6 + out) + 4 * vectors * case["d"] + 8 * t, "flops": 14.0 * n}
    n = len(case["axes"].split("+"))
    if case["kind"] == "rope":
        rows, cache = t * case["heads"] * case["dim"], 0
    else:
        rows, cache = t * case["q_heads"] * case["dim"], t * 2 * case["kv_heads"] * case["dim"]
    return {"bytes": 4 * rows + cache * (2 + 17 / 32 * 2 + 2) + t * (4 * n + 8 * (cache > 0)),
            "flops": 7.0 * (rows + cache / 2)}


# ---------------------------------------------------------------- inputs

def _rows(g, n, width):
    """bf16 activations [n][width] with a few large channels."""
    x = torch.randn((n, width), generator=g, device=DEV)
    x[:, torch.randperm(width, generator=g, device=DEV)[: width // 64]] *= 8.0
    return x.to(torch.bfloat16)


def _positions(g, case, n):
    """int32 [tokens][n]: a running position for each sequence, or places in each sequence's image or video."""
    t = torch.arange(case["tokens"], device=DEV)
    per = -(-case["tokens"] // case["seqs"])
    at = t % per
    if n == 1:
        start = torch.randint(0, case["far"] + 1, (case["seqs"],), generator=g, device=DEV)
        return (start[t // per] + at).to(torch.int32)[:, None].contiguous()
    side = math.isqrt(per if n == 2 else -(-per // 5)) + 1
    place = (at % side, at // side) if n == 2 else (at % side, at // side % side, at // side // side)
    return torch.stack(place[::-1], 1).to(torch.int32).contiguous()


def _freqs(axes, far):
    """Radians a position for each pair of channels, axis by axis."""
    base = 1e6 if far else 1e4
    return torch.cat([base ** (-torch.arange(a // 2, dtype=torch.float64) * 2 / a) for a in axes]).to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t = case["tokens"]

    def weight(n):
        return torch.rand((n,), generator=g, device=DEV) + 0.5

    def like(rows, width):
        return torch.empty((rows, width), dtype=torch.bfloat16, device=DEV)

    if case["kind"] == "norm":
        d, n = case["d"], case["samples"]
        s = dict(case=case, x=_rows(g, t, d), y=_rows(g, t, d), x_out=like(t, d), per=-(-t // n), post_w=None, pre_w=None,
                 gate=None, scale=None, shift=None)
        if case["weights"]:
            s["post_w"], s["pre_w"] = weight(d) if case["post"] != "none" else None, weight(d)
        if case["gate"]:
            s["gate"] = torch.randn((n, d), generator=g, device=DEV)
        if case["modulate"]:
            s["scale"] = 0.3 * torch.randn((n, d), generator=g, device=DEV)
            s["shift"] = 0.3 * torch.randn((n, d), generator=g, device=DEV)
        if case["out"] != "stats":
            s["h"] = like(t, d)
        else:
            s["stats"] = torch.empty((t, 2), device=DEV)
        if case["out"] == "codes":
            s["codes"] = torch.empty((t, d // 2), dtype=torch.uint8, device=DEV)
            s["scales"] = torch.empty((t, d // 32), dtype=torch.uint8, device=DEV)
            s["order"] = torch.arange(t, dtype=torch.int32, device=DEV)
        return s
    axes = tuple(int(a) for a in case["axes"].split("+"))
    s = dict(case=case, axes=axes, positions=_positions(g, case, len(axes)), freqs=_freqs(axes, case["far"]),
             weight=weight(case["dim"]) if case["norm"] else None)
    if case["kind"] == "rope":
        s["x"], s["out"] = _rows(g, t, case["heads"] * case["dim"]), like(t, case["heads"] * case["dim"])
        return s
    q, width, n, page = case["q_heads"] * case["dim"], case["kv_heads"] * case["dim"], case["slots"], case["page"]
    s["k_weight"] = weight(case["dim"]) if case["norm"] else None
    s["qkv"] = _rows(g, t, q + 2 * width)  # a fused projection: queries, keys, values
    s["q_out"] = like(t, q) if q else None
    pages = torch.randperm(n // page, generator=g, device=DEV)[: -(-t // page)]
    s["at"] = (pages[:, None] * page + torch.arange(page, device=DEV)).reshape(-1)[:t].to(torch.int32)
    if case["padded"]:  # tokens without a slot: the padding of a batch
        s["at"][torch.randperm(t, generator=g, device=DEV)[: case["padded"]]] = -1
    s["cache"] = [torch.zeros((n, w), dtype=torch.uint8, device=DEV) for w in (width // 2, width // 32) * 2]
    s["k_out"], s["v_out"] = like(t, width), like(t, width)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own(kind, state)
    return {"rope": _plain_rope, "append": _plain_append, "norm": _plain_norm}[kind](state)


def _own(kind, s):
    import w4a4_diffusion_transformer_amd as kq

    case = s["case"]
    if kind == "norm":
        norms = {"none": kq.KQ_NORM_NONE, "rms": kq.KQ_NORM_RMS, "layer": kq.KQ_NORM_LAYER}
        codes = case["out"] == "codes"
        kq.kq_residual_norm(s["x"], s["y"], s["x_out"], post=norms[case["post"]], post_weight=s["post_w"], gate=s["gate"],
                            residual_scale=case["scale"], pre=norms[case["pre"]], pre_weight=s["pre_w"],
                            mod_scale=s["scale"], mod_shift=s["shift"], tokens_per_sample=s["per"], eps=EPS,
                            h=s["h"] if case["out"] == "rows" else None, out_codes=s["codes"] if codes else None,
                            out_scales=s["scales"] if codes else None,
                            row_stats=s["stats"] if case["out"] == "stats" else None)
        if codes:
            kq.kq_cache_read(s["codes"], s["scales"], None, None, s["order"], s["h"], None)
        return {"x": s["x_out"], case["out"]: s["stats"] if case["out"] == "stats" else s["h"]}
    turn = kq.Rotation(s["positions"], s["freqs"], s["axes"], halves=case["halves"])
    norm = kq.KQ_NORM_RMS if case["norm"] else kq.KQ_NORM_NONE
    if kind == "rope":
        kq.kq_rope(s["x"], s["out"], case["heads"], rotation=turn, norm=norm, weight=s["weight"], eps=EPS)
        return s["out"]
    q, width = case["q_heads"] * case["dim"], case["kv_heads"] * case["dim"]
    kq.kq_cache_write_rope(s["qkv"][:, q:q + width], s["qkv"][:, q + width:], s["at"], *s["cache"],
                           kv_heads=case["kv_heads"], rotation=turn, norm=norm, k_weight=s["k_weight"], eps=EPS,
                           Q=s["qkv"][:, :q] if q else None, q_out=s["q_out"], q_heads=case["q_heads"],
                           q_weight=s["weight"])
    kq.kq_cache_read(*s["cache"], s["at"], s["k_out"], s["v_out"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]} if q else {"k": s["k_out"], "v": s["v_out"]}


def _bf16(x):
    """Values rounded to bf16, ties to even; float64 in one rounding (torch takes two, through float32)."""
    if x.dtype != torch.float64:
        return x.to(torch.bfloat16)
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256), e - 8).to(torch.bfloat16)


def _mx(x):
    """The values of MXFP4 of bf16 rows [..][32 n], by the OCP rules: floor of the block's exponent, nearest code."""
    b = x.float().reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    unit = torch.where(amax > 0, torch.exp2((torch.frexp(amax)[1] - 3).clamp(-126, 127).float()), 1.0)
    a = (b / unit).abs()
    borders = torch.tensor(BORDERS, device=x.device)
    code = torch.bucketize(a, borders)  # borders below a
    code = code + ((code % 2 == 1) & (a == borders[code.clamp(max=6)])).int()  # at a border: up to the even code
    y = torch.tensor(E2M1, device=x.device)[code.long()] * unit
    return torch.where(b < 0, -y, y).reshape(x.shape).to(torch.bfloat16)


def _turned(x, s, heads, weight, dtype):
    """Rows of heads, normalised and turned."""
    case, half = s["case"], sum(s["axes"]) // 2
    t, dim = x.shape[0], case["dim"]
    x = x.reshape(t, heads, dim).to(dtype)
    if case["norm"]:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.to(dtype)
    axis = torch.tensor([i for i, a in enumerate(s["axes"]) for _ in range(a // 2)], device=x.device)
    angle = s["positions"].double()[:, axis] * s["freqs"]
    c, n = torch.cos(angle).to(dtype)[:, None], torch.sin(angle).to(dtype)[:, None]
    rest = x[..., 2 * half:]
    if case["halves"]:
        a, b = x[..., :half], x[..., half:2 * half]
        return torch.cat((a * c - b * n, a * n + b * c, rest), -1).reshape(t, -1)
    a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
    return torch.cat((torch.stack((a * c - b * n, a * n + b * c), -1).flatten(-2), rest), -1).reshape(t, -1)


def _plain_rope(s):
    return _turned(s["x"], s, s["case"]["heads"], s["weight"], torch.float32).to(torch.bfloat16)


def _plain_append(s):
    case = s["case"]
    q, width = case["q_heads"] * case["dim"], case["kv_heads"] * case["dim"]
    there = (s["at"] >= 0)[:, None]
    # 64 bits: a key next to a border between two codes goes to the side that the formula gives
    k = _mx(_bf16(_turned(s["qkv"][:, q:q + width], s, case["kv_heads"], s["k_weight"], torch.float64)))
    v = _mx(s["qkv"][:, q + width:])
    out = {"k": torch.where(there, k, 0.0), "v": torch.where(there, v, 0.0)}
    if q:
        out["q"] = _turned(s["qkv"][:, :q], s, case["q_heads"], s["weight"], torch.float32).to(torch.bfloat16)
    return out


def _plain_norm(s):
    case = s["case"]
    # 64 bits as for the keys above, and for statistics, which a step of x would change
    dtype = torch.float32 if case["out"] == "rows" else torch.float64
    sample = torch.arange(case["tokens"], device=DEV) // s["per"]

    def norm(x, kind, weight):
        """(normalised, mean, 1 / deviation); sums in 64 bits."""
        mean = rstd = None
        if kind != "none":
            w = x.double()
            mean = w.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(w[:, :1])
            rstd = 1 / torch.sqrt(((w - mean) ** 2).mean(-1, keepdim=True) + EPS)
            x = (x - mean.to(dtype)) * rstd.to(dtype)
        return (x if weight is None else x * weight.to(dtype)), mean, rstd

    u = norm(s["y"].to(dtype), case["post"], s["post_w"])[0]
    if s["gate"] is not None:
        u = u * s["gate"].to(dtype)[sample]
    x = _bf16(s["x"].to(dtype) * case["scale"] + u)
    h, mean, rstd = norm(x.to(dtype), case["pre"], s["pre_w"])
    if case["out"] == "stats":
        return {"x": x, "stats": torch.cat((mean, rstd), 1).float()}
    if s["scale"] is not None:
        h = h * (1 + s["scale"].to(dtype)[sample]) + s["shift"].to(dtype)[sample]
    h = _bf16(h)
    return {"x": x, "rows": h} if case["out"] == "rows" else {"x": x, "codes": _mx(h)}


# ---------------------------------------------------------------- in 64 bits

def _exact_bf16(x):
    """Nearest bf16, ties to even, from the bits of the 64-bit values."""
    b = x.contiguous().view(torch.int64)
    kept = (b + ((1 << 44) - 1) + ((b >> 45) & 1)) & ~((1 << 45) - 1)
    return kept.view(torch.float64)


def _exact_mx(x):
    """Nearest MXFP4 values of rows in 64 bits: the block's largest power of two, then the grid's nearest multiple."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    step = torch.exp2((torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0))) - 2).clamp(-127, 127))
    y = (b / step).clamp(-6, 6)
    gap = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0)).double()
    return torch.where(amax > 0, torch.round(y / gap) * gap * step, 0.0).flatten(-2)


def _exact_turned(x, s, heads, weight):
    """Channel by channel: each with its partner, its pair's angle and the sign of the partner's share."""
    case, dim, half = s["case"], s["case"]["dim"], sum(s["axes"]) // 2
    x = x.double().unflatten(1, (heads, dim))
    if case["norm"]:
        x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / dim + EPS) * weight.double()
    out = x.clone()
    first, p = 0, 0
    for i, a in enumerate(s["axes"]):
        for p in range(first, first + a // 2):
            lo, hi = (p, p + half) if case["halves"] else (2 * p, 2 * p + 1)
            angle = (s["positions"][:, i].double() * s["freqs"][p])[:, None]
            z = torch.complex(x[..., lo], x[..., hi]) * torch.polar(torch.ones_like(angle), angle)
            out[..., lo], out[..., hi] = z.real, z.imag
        first += a // 2
    return out.flatten(1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rope":
        return _exact_turned(s["x"], s, case["heads"], s["weight"])
    if case["kind"] == "append":
        q, width = case["q_heads"] * case["dim"], case["kv_heads"] * case["dim"]
        there = (s["at"] >= 0).double()[:, None]
        k = _exact_turned(s["qkv"][:, q:q + width], s, case["kv_heads"], s["k_weight"])
        out = {"k": _exact_mx(_exact_bf16(k)) * there, "v": _exact_mx(s["qkv"][:, q + width:].double()) * there}
        if q:
            out["q"] = _exact_turned(s["qkv"][:, :q], s, case["q_heads"], s["weight"])
        return out

    def norm(x, kind, weight):
        m = x.mean(1, keepdim=True) if kind == "layer" else 0.0 * x[:, :1]
        r = (x - m).square().sum(1, keepdim=True).div(case["d"]).add(EPS).rsqrt()
        return (x - m) * r * (1.0 if weight is None else weight.double()), m, r

    def per_row(v):
        return v.double().repeat_interleave(s["per"], 0)[: case["tokens"]]

    u = s["y"].double() if case["post"] == "none" else norm(s["y"].double(), case["post"], s["post_w"])[0]
    x = case["scale"] * s["x"].double() + (u * per_row(s["gate"]) if case["gate"] else u)
    h, m, r = norm(_exact_bf16(x), case["pre"], s["pre_w"])
    if case["out"] == "stats":
        return {"x": x, "stats": torch.cat((m, r), 1)}
    if case["modulate"]:
        h = h * (1 + per_row(s["scale"])) + per_row(s["shift"])
    return {"x": x, "rows": h} if case["out"] == "rows" else {"x": x, "codes": _exact_mx(_exact_bf16(h))}
