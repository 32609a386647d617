"""Plain 64-bit forms of the cache, attention and epilogue operators, on the CPU."""
import math

import numpy as np
import torch

import oracle


def values(codes, scales) -> torch.Tensor:
    """The values of MXFP4 rows (uint8 tensors) in float64."""
    return torch.from_numpy(oracle.dequant_rows(codes.cpu().numpy(), scales.cpu().numpy()).astype(np.float64))


def quantize(x: torch.Tensor):
    """Plain MXFP4 of bf16 rows: (codes, scales) uint8."""
    r = oracle.quantize_rows(oracle.PLAIN, x.contiguous().view(torch.int16).numpy().view(np.uint16))
    return torch.from_numpy(r["codes"]), torch.from_numpy(r["scales"])


def bf16(shape, seed, scale=1.0) -> torch.Tensor:
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def slots_of(table, b, n, page_size, n_slots):
    """Slot of each of sequence b's first n keys, -1 where its page is not in the cache."""
    j = torch.arange(n)
    page = table[b].long()[j // page_size]
    return torch.where((page >= 0) & (page < n_slots // page_size), page * page_size + j % page_size, -1)


def attention(q, cache, kv_len, table, page_size, q_heads, kv_heads, q_start, scale=None, causal=False):
    """Attention in float64 and the bound on a kernel's error.

    q [rows, q_heads * dim] bf16; cache four uint8 pools; q_start a list of batch + 1 rows.  Returns out, lse, the
    bounds on their errors, and which rows belong to a sequence.

    The bound of a kernel that keeps scores, maxima and sums in fp32, rounds the probabilities and the output once to
    bf16 (half a step, 2^-8 relative) and nothing else: with E the largest error of a score (a dot product of dim fp32
    terms, each rounding at most 2^-24 of the sum of magnitudes, and the exponent's own roundings, some 2^-22 of its
    size), a probability is off by a factor within exp(E) (1 + 2^-8), their sum of n terms by exp(E) (1 + n 2^-24).
    """
    kc, ks, vc, vs = cache
    rows, dim, group = q.shape[0], q.shape[1] // q_heads, q_heads // kv_heads
    scale = dim ** -0.5 if scale is None else scale
    out = torch.zeros((rows, q_heads, dim), dtype=torch.float64)
    lse = torch.full((rows, q_heads), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    owned = torch.zeros(rows, dtype=torch.bool)
    for b in range(len(q_start) - 1):
        r0, r1, n = q_start[b], q_start[b + 1], int(kv_len[b])
        owned[r0:r1] = True
        at = slots_of(table, b, n, page_size, kc.shape[0])
        there = at >= 0
        take = at.clamp(min=0)
        k = torch.where(there[:, None], values(kc[take], ks[take]), 0.0).unflatten(1, (kv_heads, dim))
        v = torch.where(there[:, None], values(vc[take], vs[take]), 0.0).unflatten(1, (kv_heads, dim))
        seen = there[None, :].expand(r1 - r0, n)
        if causal:
            seen = seen & (torch.arange(n)[None, :] <= n - (r1 - r0) + torch.arange(r1 - r0)[:, None])
        for h in range(q_heads):
            x = q[r0:r1, h * dim:(h + 1) * dim].double()
            kh, vh = k[:, h // group], v[:, h // group]
            s = (x @ kh.T * scale).masked_fill(~seen, -math.inf)
            size = ((x.abs() @ kh.T.abs()) * scale).masked_fill(~seen, 0.0)
            lse[r0:r1, h] = torch.logsumexp(s, 1) if n else -math.inf
            some = seen.any(1)
            p = torch.where(some[:, None], torch.exp(s - lse[r0:r1, h, None]), 0.0) if n else s
            out[r0:r1, h] = p @ vh
            mag = p @ vh.abs()
            err = ((dim + 8) * 2.0 ** -24 * size.amax(1) + 2.0 ** -21 * (1 + size.amax(1))) if n else torch.zeros(r1 - r0)
            e = (err + n * 2.0 ** -24)[:, None]
            tol[r0:r1, h] = mag * (2 * e + 2.0 ** -8) + 2.0 ** -8 * out[r0:r1, h].abs() * (1 + 2 * e) + 1e-30
            tol_lse[r0:r1, h] = torch.where(some, e[:, 0] + 2.0 ** -22 * lse[r0:r1, h].abs(), 0.0)
    return out.flatten(1), lse, tol.flatten(1), tol_lse, owned


def check_attention(got, got_lse, ref):
    """Asserts a kernel's out (bf16) and lse against attention()'s result on the rows that belong to a sequence."""
    out, lse, tol, tol_lse, owned = ref
    got, got_lse = got.cpu().double(), got_lse.cpu().double()
    assert torch.isfinite(got[owned]).all()
    over = ((got - out).abs() - tol)[owned]
    assert over.max().item() <= 0 if over.numel() else True, f"out: {over.max().item():.3g} past the bound"
    empty = torch.isinf(lse) & owned[:, None]
    assert torch.equal(torch.isneginf(got_lse) & owned[:, None], empty)
    fine = ~torch.isinf(lse) & owned[:, None]
    over = ((got_lse - lse).abs() - tol_lse)[fine]
    assert over.max().item() <= 0 if over.numel() else True, f"lse: {over.max().item():.3g} past the bound"


def act(x, name):
    if name == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    if name == "gelu_erf":
        return 0.5 * x * torch.special.erfc(-x / math.sqrt(2))
    return x * torch.sigmoid(x) if name == "silu" else x


def gemm(a, a_s, b, b_s, bias, name, gate, rows_per_sample, residual):
    """The product with its epilogue in float64, and the bound on an fp32 kernel's error: the sums of K exact products
    (K roundings of at most 2^-24 of the sum of magnitudes), activations of slope at most 1.13 with an error of 2^-21
    max(|x|, 1), and three more roundings of 2^-24."""
    A, B = values(a, a_s), values(b, b_s)
    x = A @ B.T
    err = (A.shape[1] * 2.0 ** -24) * (A.abs() @ B.abs().T)
    if bias is not None:
        x = x + bias.double()
        err = err + 2.0 ** -24 * x.abs()
    if name != "none":
        err = 1.13 * err + 2.0 ** -21 * x.abs().clamp(min=1)
    y = act(x, name)
    if gate is not None:
        g = gate.double().repeat_interleave(rows_per_sample, 0)[: y.shape[0]]
        y = y * g
        err = err * g.abs() + 2.0 ** -24 * y.abs()
    if residual is not None:
        y = y + residual.double()
        err = err + 2.0 ** -24 * y.abs()
    return y, err * (1 + 2.0 ** -10) + 1e-30
