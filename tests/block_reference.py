"""Plain 64-bit forms, on the CPU, of the rotary, rotated cache-append and residual-norm operators, each with the bound
on what a kernel that works in fp64 and rounds once to bf16 may give."""
import torch

import cache_reference as cache

SLACK = 2.0 ** -40  # fp64 kernels: a few dozen roundings of 2^-53, and series that end below 2^-44


def rounded(x: torch.Tensor) -> torch.Tensor:
    """float64 values rounded once to bf16, ties to even (a conversion by way of fp32 rounds twice)."""
    m, e = torch.frexp(x)
    e = torch.clamp(e, min=-125)  # below 2^-126 the step stays 2^-133
    step = torch.ldexp(torch.ones_like(x), e - 8)
    return torch.where(torch.isfinite(x), torch.round(x / step) * step, x)


def between(want: torch.Tensor, slack: torch.Tensor):
    """What may come out of a value known to `slack`: the roundings of both ends, equal unless a tie lies between."""
    return rounded(want - slack), rounded(want + slack)


def check(got: torch.Tensor, want: torch.Tensor, slack: torch.Tensor, what: str = "") -> None:
    lo, hi = between(want, slack)
    got = got.cpu().double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities"
    fine = ~(nan | inf)
    off = ((got < lo) | (got > hi)) & fine
    assert not off.any(), f"{what}: {int(off.sum())} of {off.numel()} off, first {got[off][0]} for {want[off][0]}"


def rope(x, heads, rotation=None, rms=False, weight=None, eps=1e-6):
    """(values, slack) of bf16 rows x [tokens, heads * dim]; rotation: (positions, freqs, axis_dims, halves)."""
    n = x.double().unflatten(1, (heads, -1))
    if rms:
        n = n * (1 / torch.sqrt((n * n).sum(-1, keepdim=True) / n.shape[-1] + eps))
        if weight is not None:
            n = n * weight.double()
    y, size = n.clone(), n.abs()
    far = torch.zeros_like(n)  # error of angles
    if rotation is not None:
        positions, freqs, dims, halves = rotation
        half, p = sum(dims) // 2, 0
        for axis, d in enumerate(dims):
            for _ in range(d // 2):
                i, j = (p, p + half) if halves else (2 * p, 2 * p + 1)
                angle = (positions[:, axis].double() * freqs[p])[:, None]
                u, v, c, s = n[..., i], n[..., j], torch.cos(angle), torch.sin(angle)
                y[..., i], y[..., j] = u * c - v * s, u * s + v * c
                for k in (i, j):
                    size[..., k] = u.abs() + v.abs()
                    far[..., k] = (u.abs() + v.abs()) * angle.abs() * 2.0 ** -51
                p += 1
    return y.flatten(1), (size * SLACK + far).flatten(1)


def norm(x, kind, eps):
    """(normalised rows, mean, 1 / deviation) in float64; kind 0 none, 1 RMS, 2 layer."""
    if kind == 0:
        return x, None, None
    mean = x.mean(1, keepdim=True) if kind == 2 else torch.zeros_like(x[:, :1])
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    return (x - mean) * rstd, mean, rstd


def per_row(v, per, tokens):
    return v.double().repeat_interleave(per, 0)[:tokens]


def residual(x, y, post=0, post_weight=None, gate=None, scale=1.0, per=None, eps=1e-6):
    """(x', slack) of the stream."""
    per = x.shape[0] if per is None else per
    raw, mean, rstd = norm(y.double(), post, eps)
    size = raw.abs() if mean is None else raw.abs() + (mean * rstd).abs()
    u = raw
    for f in (None if post_weight is None else post_weight.double(), None if gate is None else per_row(gate, per, x.shape[0])):
        if f is not None:
            u, size = u * f, size * f.abs()
    return scale * x.double() + u, (abs(scale) * x.double().abs() + size) * SLACK


def following(x, pre=0, pre_weight=None, mod_scale=None, mod_shift=None, per=None, eps=1e-6):
    """(h, slack, mean, rstd) of the stored stream x (bf16)."""
    per = x.shape[0] if per is None else per
    h, mean, rstd = norm(x.double(), pre, eps)
    size = h.abs() if mean is None else h.abs() + (mean * rstd).abs()
    if pre_weight is not None:
        h, size = h * pre_weight.double(), size * pre_weight.double().abs()
    if mod_scale is not None:
        f = 1 + per_row(mod_scale, per, x.shape[0])
        h, size = h * f, size * f.abs()
    if mod_shift is not None:
        f = per_row(mod_shift, per, x.shape[0])
        h, size = h + f, size + f.abs()
    return h, size * SLACK, mean, rstd


def check_codes(codes, scales, rows, what=""):
    """Codes and scales are the plain MXFP4 of bf16 rows."""
    want = cache.quantize(rows.cpu())
    assert torch.equal(codes.cpu(), want[0]) and torch.equal(scales.cpu(), want[1]), f"{what}: codes of other values"
