"""The cached-attention and epilogue operators: what is timed, and their plain forms.

Four operators of a W4A4 transformer step, each with cases over the sizes it meets:
  * kq_cache_write  quantises new key and value rows to MXFP4 and writes them to their slots of a paged cache;
  * kq_cache_read   gathers slots of that cache and gives back the bf16 values they stand for;
  * kq_attention_mx attention of bf16 queries over the 4-bit cache (cross attention, prompts, single tokens);
  * kq_gemm_mx_ex   the MXFP4 product with bias, activation, gate and residual in its epilogue.

`own = False` computes them with elementary torch operations in 32 bits; `own = True` calls the library.
"""
import math

import torch

own = False

DEV = "cuda:0"

# E2M1 values by code (bit 3 is the sign), and E2M1 magnitudes' rounding borders: a value above
# LOW[i], or at UP[i] and above, has the next code (ties go to the even code).
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
LOW = (0.25, 1.25, 2.5, 5.0)
UP = (0.75, 1.75, 3.5)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # eight sequences that each take one new token: the append of a decode step, all latency
        dict(name="write_step", kind="write", tokens=8, heads=8, dim=128, slots=4096, page=64, padded=1),
        # a long prompt's keys and values, rows of a fused projection, an odd token count
        dict(name="write_prompt", kind="write", tokens=40961, heads=8, dim=128, slots=65536, page=64, padded=0),
        # the text states of eight prompts of 300 tokens at the 1152-wide diffusion transformer
        dict(name="read_text", kind="read", tokens=2400, heads=16, dim=72, slots=4096, page=100, padded=37),
        # every page of a large cache gathered in order for a product in bf16
        dict(name="read_long", kind="read", tokens=65536, heads=8, dim=128, slots=81920, page=64, padded=0),
        # one sequence, one new token, a short context: the smallest decode step
        dict(name="attn_token", kind="attn", batch=1, q=1, ragged=False, kv_min=1023, kv_max=1023, q_heads=32,
             kv_heads=8, dim=128, page=64, table=True, causal=True),
        # a decode batch of contexts between nothing (a padded entry) and 16384, grouped heads
        dict(name="attn_tokens", kind="attn", batch=32, q=1, ragged=False, kv_min=0, kv_max=16384, q_heads=32,
             kv_heads=8, dim=128, page=64, table=True, causal=True),
        # image tokens over text states of up to 300 tokens, 16 heads of 72 (the 1152-wide transformer), guidance batch
        dict(name="attn_cross", kind="attn", batch=8, q=4096, ragged=False, kv_min=11, kv_max=300, q_heads=16,
             kv_heads=16, dim=72, page=300, table=False, causal=False),
        # joint attention of 4608 image and text tokens over a cache of 5120, heads of 128
        dict(name="attn_joint", kind="attn", batch=1, q=4608, ragged=False, kv_min=5120, kv_max=5120, q_heads=16,
             kv_heads=16, dim=128, page=64, table=True, causal=False),
        # chunks of four prompts, ragged, each over what is cached before it
        dict(name="attn_prompt", kind="attn", batch=4, q=1777, ragged=True, kv_min=1800, kv_max=8001, q_heads=32,
             kv_heads=8, dim=128, page=64, table=True, causal=True),
        # the modulation vectors (six of 1152) of a guidance pair: a product of two rows, fp32 out
        dict(name="gemm_modulation", kind="gemm", m=2, n=6912, k=1152, bias=True, act="none", gate=False,
             residual=False, fp32=True),
        # the first MLP layer of the 1152-wide transformer with its activation
        dict(name="gemm_mlp_in", kind="gemm", m=8192, n=4608, k=1152, bias=True, act="gelu_tanh", gate=False,
             residual=False, fp32=False),
        # the second MLP layer at the 2240-wide transformer, gated into the residual stream
        dict(name="gemm_mlp_out", kind="gemm", m=4096, n=2240, k=5600, bias=True, act="none", gate=True,
             residual=True, fp32=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("write", "read", "attn", "attn", "attn", "gemm"))
    if kind == "gemm":
        while True:
            c = dict(kind="gemm", m=_log(rng, 1, 8192), n=_log(rng, 64, 9216), k=32 * _log(rng, 2, 384),
                     bias=rng.random() < 0.8, act=rng.choice(("none", "gelu_tanh", "gelu_erf", "silu")),
                     gate=rng.random() < 0.5, residual=rng.random() < 0.5, fp32=rng.random() < 0.3)
            if c["m"] * c["n"] * c["k"] <= 8192 * 4608 * 1152:
                return c
    dim = rng.choice((32, 64, 72, 80, 96, 112, 128))
    heads = rng.choice([h for h in (1, 2, 4, 5, 8, 12, 16, 20) if h * dim % 32 == 0])
    if kind in ("write", "read"):
        tokens = _log(rng, 1, 65536)
        while tokens * heads * dim > 40000 * 1024:
            tokens = _log(rng, 1, 65536)
        page = rng.choice((16, 50, 64, 128, 300))
        return dict(kind=kind, tokens=tokens, heads=heads, dim=dim, page=page,
                    slots=page * (-(-tokens // page) + rng.randint(1, 40)), padded=rng.choice((0, min(tokens - 1, 5))))
    form = rng.choice(("tokens", "cross", "prompt"))
    group = rng.choice((1, 2, 4, 8))
    while True:
        batch = _log(rng, 1, 32 if form == "tokens" else 8)
        q = 1 if form == "tokens" else _log(rng, 2, 4608)
        kv = _log(rng, 1, 512 if form == "cross" else 16384 if form == "tokens" else 8192)
        scores = batch * heads * group * q * kv
        if scores <= 4 * 32 * 1777 * 8001 and batch * kv * heads * dim <= 32 * 16384 * 1024 and scores * dim <= 16 * 4608 * 5120 * 128:
            break
    return dict(kind="attn", batch=batch, q=q, ragged=form == "prompt", kv_min=rng.randint(0, kv), kv_max=kv,
                q_heads=heads * group, kv_heads=heads, dim=dim, page=rng.choice((16, 50, 64, 128)),
                table=rng.random() < 0.7, causal=form != "cross")


def _lengths(case):
    """Each sequence's number of cached tokens and of queries."""
    n = case["batch"]
    step = next(s for s in (5, 7, 11, 13) if math.gcd(s, n) == 1)
    kv = [case["kv_max"] if n == 1 else case["kv_min"] + (case["kv_max"] - case["kv_min"]) * ((step * i + 3) % n) // (n - 1)
          for i in range(n)]
    q = [max(1, case["q"] - (case["q"] // 2) * i // n) if case["ragged"] else case["q"] for i in range(n)]
    return kv, q


def work(case):
    if case["kind"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        out = m * n * (4 if case["fp32"] else 2)
        extra = 4 * n * case["bias"] + 4 * n * _samples(m)[0] * case["gate"] + 2 * m * n * case["residual"]
        return {"bytes": (m + n) * k * 17 / 32 + out + extra, "flops": 2.0 * m * n * k}
    width = case.get("heads", case.get("kv_heads")) * case["dim"]
    if case["kind"] == "write":  # the rows in, the cache's bytes out, and the values read back out
        return {"bytes": case["tokens"] * (2 * width * (2 + 17 / 32 + 2) + 4), "flops": 0}
    if case["kind"] == "read":
        return {"bytes": case["tokens"] * (2 * width * (17 / 32 + 2) + 4), "flops": 0}
    kv, q = _lengths(case)
    pairs = 0
    for n, m in zip(kv, q):  # causal: query i of m sees the first n - m + 1 + i keys
        pairs += sum(max(0, n - m + 1 + i) for i in range(m)) if case["causal"] else n * m
    rows = sum(q)
    qo = rows * case["q_heads"] * case["dim"] * 2
    return {"bytes": sum(kv) * width * 2 * 17 / 32 + 2 * qo + 4 * rows * case["q_heads"],
            "flops": 4.0 * pairs * case["q_heads"] * case["dim"]}


# ---------------------------------------------------------------- inputs

def _grid():
    """The grid's values and borders on the GPU."""
    return {k: torch.tensor(v, device=DEV) for k, v in (("values", E2M1), ("low", LOW), ("up", UP))}


def _mx(x, grid):
    """MXFP4 of fp32 rows [.., 32 n]: (codes, scales), OCP MX rules."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    byte = torch.where(amax > 0, (torch.frexp(amax)[1] - 1 - 2 + 127).clamp(0, 254), 0)
    y = b * ((254 - byte) << 23).view(torch.float32).unsqueeze(-1)  # b / 2^(byte - 127)
    a = y.abs()
    below = torch.bucketize(a, grid["low"])  # how many borders of LOW are under a
    upto = torch.bucketize(a, grid["up"], right=True)  # how many of UP are at it or under it
    code = (8 * (y < 0) + below + upto).to(torch.uint8).reshape(*x.shape[:-1], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), byte.to(torch.uint8)


def _values(codes, scales, grid):
    """The fp32 values of MXFP4 rows."""
    v = torch.stack((grid["values"][(codes & 15).int()], grid["values"][(codes >> 4).int()]), -1).reshape(*codes.shape[:-1], -1, 32)
    s = torch.where(scales > 0, scales.int() << 23, 0x00400000).view(torch.float32)  # 2^(byte - 127)
    return (v * s.unsqueeze(-1)).reshape(*codes.shape[:-1], -1)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(g, n, width):
    """bf16 activations [n][width] with a few large channels, as keys have them."""
    x = torch.randn((n, width), generator=g, device=DEV)
    x[:, torch.randperm(width, generator=g, device=DEV)[: width // 64]] *= 8.0
    return x.to(torch.bfloat16)


def _samples(m):
    """How many samples m rows are, and the rows of each: the guidance batch."""
    n = 2 if m % 2 == 0 else 1
    return n, m // n


def prepare(case, seed):
    g, grid = _gen(seed), _grid()
    if case["kind"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        ac, asc = _mx(torch.randn((m, k), generator=g, device=DEV).to(torch.bfloat16).float(), grid)
        bc, bsc = _mx((torch.randn((n, k), generator=g, device=DEV) * k ** -0.5).to(torch.bfloat16).float(), grid)
        return dict(case=case, grid=grid, a=ac, a_s=asc, b=bc, b_s=bsc,
                    bias=torch.randn((n,), generator=g, device=DEV) if case["bias"] else None,
                    gate=torch.randn((_samples(m)[0], n), generator=g, device=DEV) if case["gate"] else None,
                    residual=torch.randn((m, n), generator=g, device=DEV).to(torch.bfloat16) if case["residual"] else None,
                    y=torch.empty((m, n), dtype=torch.float32 if case["fp32"] else torch.bfloat16, device=DEV))
    if case["kind"] in ("write", "read"):
        t, width, n = case["tokens"], case["heads"] * case["dim"], case["slots"]
        pages = torch.randperm(n // case["page"], generator=g, device=DEV)[: -(-t // case["page"])]
        at = (pages[:, None] * case["page"] + torch.arange(case["page"], device=DEV)).reshape(-1)[:t].to(torch.int32)
        if case["padded"]:  # tokens without a slot: the padding of a batch
            at[torch.randperm(t, generator=g, device=DEV)[: case["padded"]]] = -1
        # one row more than the cache has: where the plain form puts what has no slot
        kc, ks = _mx(_rows(g, n + 1, width).float(), grid)
        vc, vs = _mx(_rows(g, n + 1, width).float(), grid)
        s = dict(case=case, grid=grid, slots=at, k_codes=kc, k_scales=ks, v_codes=vc, v_scales=vs,
                 k_out=torch.empty((t, width), dtype=torch.bfloat16, device=DEV),
                 v_out=torch.empty((t, width), dtype=torch.bfloat16, device=DEV))
        s["cache"] = [t[:n] for t in (kc, ks, vc, vs)]
        if case["kind"] == "write":
            s["kv"] = _rows(g, t, 2 * width)  # a fused projection: keys, then values
        return s
    kv, q = _lengths(case)
    width, page = case["kv_heads"] * case["dim"], case["page"]
    per = -(-max(kv + [1]) // page)  # pages of a sequence
    pages = case["batch"] * per
    kc, ks = _mx(_rows(g, pages * page, width).float(), grid)
    vc, vs = _mx(_rows(g, pages * page, width).float(), grid)
    table = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).reshape(case["batch"], per)
    rows = sum(q)
    starts = [sum(q[:i]) for i in range(case["batch"] + 1)]
    qs = torch.randn((rows, case["q_heads"] * case["dim"]), generator=g, device=DEV).to(torch.bfloat16)
    return dict(case=case, grid=grid, q=qs, k_codes=kc, k_scales=ks, v_codes=vc, v_scales=vs, per=per,
                table=table if case["table"] else None,
                kv_len=torch.tensor(kv, dtype=torch.int32, device=DEV),
                q_start=torch.tensor(starts, dtype=torch.int32, device=DEV) if case["ragged"] else None, max_q=max(q),
                out=torch.empty_like(qs), lse=torch.empty((rows, case["q_heads"]), device=DEV))


# ---------------------------------------------------------------- one pass

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own(kind, state)
    return {"gemm": _plain_gemm, "write": _plain_write, "read": _plain_read, "attn": _plain_attn}[kind](state)


def _own(kind, s):
    import w4a4_diffusion_transformer_amd as kq

    case = s["case"]
    if kind == "gemm":
        act = {"none": kq.KQ_ACT_NONE, "gelu_tanh": kq.KQ_ACT_GELU_TANH, "gelu_erf": kq.KQ_ACT_GELU_ERF,
               "silu": kq.KQ_ACT_SILU}[case["act"]]
        kq.kq_gemm_mx_ex(s["a"], s["a_s"], s["b"], s["b_s"], bias=s["bias"], act=act, gate=s["gate"],
                         rows_per_sample=_samples(case["m"])[1], residual=s["residual"],
                         y_f32=s["y"] if case["fp32"] else None, y_bf16=None if case["fp32"] else s["y"])
        return s["y"]
    if kind == "attn":
        kq.kq_attention_mx(s["q"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["kv_len"], s["out"],
                           case["q_heads"], case["kv_heads"], page_size=case["page"], pages_per_seq=s["per"],
                           page_table=s["table"], q_start=s["q_start"], max_q=s["max_q"], causal=case["causal"],
                           lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if kind == "write":
        width = case["heads"] * case["dim"]
        kq.kq_cache_write(s["kv"][:, :width], s["kv"][:, width:], s["slots"], *s["cache"])
    kq.kq_cache_read(*s["cache"], s["slots"], s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_read(s):
    n = s["case"]["slots"]
    at = s["slots"].long()
    there = (at >= 0) & (at < n)
    at = torch.where(there, at, n)

    def values(codes, scales):
        return torch.where(there[:, None], _values(codes[at], scales[at], s["grid"]), 0.0).to(torch.bfloat16)

    return {"k": values(s["k_codes"], s["k_scales"]), "v": values(s["v_codes"], s["v_scales"])}


def _plain_write(s):
    n, width = s["case"]["slots"], s["case"]["heads"] * s["case"]["dim"]
    at = s["slots"].long()
    at = torch.where((at >= 0) & (at < n), at, n)  # row n takes what has no slot
    kc, ks = _mx(s["kv"][:, :width].float(), s["grid"])
    vc, vs = _mx(s["kv"][:, width:].float(), s["grid"])
    s["k_codes"][at], s["k_scales"][at] = kc, ks
    s["v_codes"][at], s["v_scales"][at] = vc, vs
    return _plain_read(s)


def _plain_gemm(s):
    case = s["case"]
    y = torch.matmul(_values(s["a"], s["a_s"], s["grid"]), _values(s["b"], s["b_s"], s["grid"]).t())
    if s["bias"] is not None:
        y = y + s["bias"]
    if case["act"] == "gelu_tanh":  # y (1 + tanh(u)) / 2 = y / (1 + exp(-2 u))
        y = y / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    elif case["act"] == "gelu_erf":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif case["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    if s["gate"] is not None:
        n, rows = _samples(case["m"])
        y = (y.reshape(n, rows, -1) * s["gate"][:, None]).reshape(n * rows, -1)
    if s["residual"] is not None:
        y = s["residual"].float() + y
    return y if case["fp32"] else y.to(torch.bfloat16)


def _plain_attn(s):
    case = s["case"]
    b, hq, hk, d, page, per = case["batch"], case["q_heads"], case["kv_heads"], case["dim"], case["page"], s["per"]
    rows, mq, group = s["q"].shape[0], s["max_q"], hq // hk
    nk = per * page
    table = s["table"].long() if s["table"] is not None else torch.arange(b * per, device=DEV).reshape(b, per)
    at = (table[:, :, None] * page + torch.arange(page, device=DEV)).reshape(b, nk)
    key = torch.arange(nk, device=DEV)
    seen = key < s["kv_len"][:, None]  # [b][nk]

    def heads(codes, scales):  # [b][hk][nk][d]
        v = torch.where(seen[..., None], _values(codes[at], scales[at], s["grid"]), 0.0)
        return v.reshape(b, nk, hk, d).transpose(1, 2).contiguous()

    k, v = heads(s["k_codes"], s["k_scales"]), heads(s["v_codes"], s["v_scales"])
    i = torch.arange(mq, device=DEV)
    if s["q_start"] is None:
        first = torch.arange(b, device=DEV) * mq
        count = torch.full((b,), mq, device=DEV)
    else:
        first, count = s["q_start"][:-1].long(), (s["q_start"][1:] - s["q_start"][:-1]).long()
    row = torch.where(i < count[:, None], first[:, None] + i, rows)  # [b][mq]; row `rows` is no query
    q = torch.cat((s["q"], s["q"].new_zeros((1, hq * d))))[row].float()
    q = q.reshape(b, mq, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, group * mq, d)
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) * (1 / math.sqrt(d))
    score = score.reshape(b, hk, group, mq, nk)
    if case["causal"]:
        upto = s["kv_len"][:, None] - count[:, None] + i  # [b][mq]: the last key a query sees
        seen = seen[:, None] & (key <= upto[..., None])  # [b][mq][nk]
    else:
        seen = seen[:, None]
    score = torch.where(seen[:, None, None], score, -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -torch.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(b, hk, group * mq, nk), v).reshape(b, hk, group, mq, d) / torch.where(total > 0, total, 1.0)
    lse = (torch.log(total) + top).squeeze(-1)  # nothing seen: -inf
    out = torch.empty((rows + 1, hq * d), dtype=torch.bfloat16, device=DEV)
    out[row] = o.permute(0, 3, 1, 2, 4).reshape(b, mq, hq * d).to(torch.bfloat16)
    lses = torch.empty((rows + 1, hq), device=DEV)
    lses[row] = lse.permute(0, 3, 1, 2).reshape(b, mq, hq)
    return {"out": out[:rows], "lse": lses[:rows]}


# ---------------------------------------------------------------- in 64 bits

def _exact_values(codes, scales):
    """The values of MXFP4 rows in 64 bits: (-1)^s * m * 2^(byte - 127), from the format's bit fields."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    e, m = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((e - 1).double()))
    sign = torch.where(c >= 8, -1.0, 1.0).double()
    return sign * mag * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _exact_mx(x):
    """Nearest MXFP4 values of rows in 64 bits: the scale from the block's largest exponent, then the grid's nearest value."""
    b = x.double().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    step = torch.exp2((torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0))) - 2).clamp(-127, 127))
    y = (b / step).clamp(-6, 6)
    # the grid's spacing: 1/2 below 2, 1 below 4, 2 above; round() takes ties to the even multiple
    gap = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0)).double()
    return torch.where(amax > 0, torch.round(y / gap) * gap * step, 0.0).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "gemm":
        y = _exact_values(s["a"], s["a_s"]) @ _exact_values(s["b"], s["b_s"]).t()
        if case["bias"]:
            y += s["bias"].double()
        if case["act"] == "gelu_tanh":
            y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
        elif case["act"] == "gelu_erf":
            y = 0.5 * y * torch.special.erfc(-y / math.sqrt(2))
        elif case["act"] == "silu":
            y = y * torch.sigmoid(y)
        if case["gate"]:
            y = y * s["gate"].double().repeat_interleave(_samples(case["m"])[1], 0)
        return y + s["residual"].double() if case["residual"] else y
    if case["kind"] in ("write", "read"):
        width = case["heads"] * case["dim"]
        there = (s["slots"] >= 0)[:, None]
        if case["kind"] == "write":
            new = _exact_mx(s["kv"])
            return {"k": torch.where(there, new[:, :width], 0.0), "v": torch.where(there, new[:, width:], 0.0)}
        at = s["slots"].clamp(min=0).long()
        return {"k": torch.where(there, _exact_values(s["k_codes"][at], s["k_scales"][at]), 0.0),
                "v": torch.where(there, _exact_values(s["v_codes"][at], s["v_scales"][at]), 0.0)}
    kv, q = _lengths(case)
    hq, hk, d, page, per = case["q_heads"], case["kv_heads"], case["dim"], case["page"], s["per"]
    out = torch.zeros((sum(q), hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((sum(q), hq), -torch.inf, dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, m) in enumerate(zip(kv, q)):
        if n:
            pages = s["table"][b].long() if case["table"] else torch.arange(per, device=DEV) + b * per
            slot = (pages[:, None] * page + torch.arange(page, device=DEV)).flatten()[:n]
            k = _exact_values(s["k_codes"][slot], s["k_scales"][slot]).unflatten(1, (hk, d))
            v = _exact_values(s["v_codes"][slot], s["v_scales"][slot]).unflatten(1, (hk, d))
            for h in range(hq):
                t = s["q"][at:at + m, h * d:(h + 1) * d].double() @ k[:, h * hk // hq].t() / math.sqrt(d)
                if case["causal"]:
                    t = t.masked_fill(torch.ones_like(t, dtype=torch.bool).triu(n - m + 1), -torch.inf)
                l = torch.logsumexp(t, 1)
                lse[at:at + m, h] = l
                p = torch.exp(t - torch.where(l.isinf(), 0.0, l)[:, None])
                out[at:at + m, h] = p @ v[:, h * hk // hq]
        at += m
    return {"out": out.flatten(1), "lse": lse}
