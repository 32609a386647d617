"""Edges of the residual stream's norms on an MI355X (through the C ABI): sums that cancel, values that are not finite and
missing parts, at the row counts and widths that take each of the kernel's forms, with such rows beside others."""
import pytest
import torch

import block_reference as ref
from test_gpu_residual_norm import run_and_check, same_stats

kq = pytest.importorskip("w4a4_diffusion_transformer_amd")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    kq.lib()


# Several rows a wave, with a piece of some lanes missing; a row a wave; a row a workgroup with one and with two pieces a
# lane; rows read again. Of 96, 1152 and 2240 channels the reciprocal times the width is 1 in 64 bits, of the others not.
FORMS = [(17003, 96), (1801, 1568), (9001, 1152), (2051, 2240), (5, 3136), (5, 12544), (5, 16864)]


def rows(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(torch.bfloat16)


def norm_of(x, pre, eps):
    """(h, codes, scales, statistics) of the stream as it is."""
    tokens, d = x.shape
    xs = x.to(DEV)
    h, stats, (codes, scales) = torch.empty_like(xs), torch.empty((tokens, 2), device=DEV), kq.alloc_outputs(xs)
    kq.kq_residual_norm(xs, None, None, pre=pre, eps=eps, h=h, out_codes=codes, out_scales=scales, row_stats=stats)
    return h.cpu(), codes.cpu(), scales.cpu(), stats, xs


@pytest.mark.parametrize("tokens,d", FORMS)
def test_rows_of_one_value_are_their_mean(tokens, d):
    """Every third row holds one value: the mean is that value, so h is 0 (with eps 0: 0 / 0), its codes are those of
    zeros, and the statistics are kq_row_stats', bit for bit."""
    x = rows((tokens, d), d)
    values = torch.tensor([1.0, 10100.0, -3e38, 2.0 ** -120, 5.0, -0.1171875]).to(torch.bfloat16)
    one = torch.arange(tokens) % 3 == 1
    x[one] = values[torch.arange(int(one.sum())) % len(values)][:, None].expand(-1, d)
    for eps in (1e-6, 0.0):
        h, codes, scales, stats, xs = norm_of(x, kq.KQ_NORM_LAYER, eps)
        if eps:
            assert not h[one].any()
            ref.check_codes(codes, scales, h)
        else:
            assert torch.isnan(h[one]).all()
        assert torch.isfinite(h[~one]).all()
        again = kq.kq_row_stats(xs, eps, torch.empty_like(stats))
        assert torch.equal(again[one], stats[one])
        want, slack, *_ = ref.following(x[~one], 2, eps=eps)
        ref.check(h[~one], want, slack)


@pytest.mark.parametrize("tokens,d", FORMS)
def test_a_block_of_one_value_adds_nothing(tokens, d):
    """The same before the sum: the stream is the scaled stream."""
    x, y = rows((tokens, d), 1), rows((tokens, 1), 2, 300.0).expand(-1, d).contiguous()
    xs = x.to(DEV)
    out = torch.empty_like(xs)
    kq.kq_residual_norm(xs, y.to(DEV), out, post=kq.KQ_NORM_LAYER, residual_scale=0.5)
    assert torch.equal(out.cpu(), (x.float() * 0.5).to(torch.bfloat16))


@pytest.mark.parametrize("tokens,d", [(17003, 96), (4801, 1056), (9001, 1152), (2051, 2208), (5, 3168), (5, 12576), (5, 16896)])
def test_blocks_at_the_mean_of_a_row(tokens, d):
    """Rows whose middle third is exactly their mean (2, 3, 4 or -250, 3, 256 times a power of two): h is 0
    there, and so are its codes."""
    third = d // 3
    assert third % 32 == 0
    x = torch.empty((tokens, 3, third))
    x[:, 0], x[:, 1], x[:, 2] = 2.0, 3.0, 4.0
    x[1::2, 0], x[1::2, 2] = -250.0, 256.0
    x = (x.flatten(1) * torch.exp2(torch.arange(tokens) % 7 - 3.0)[:, None]).to(torch.bfloat16)
    h, codes, scales, *_ = norm_of(x, kq.KQ_NORM_LAYER, 1e-6)
    assert not h[:, third:2 * third].any()
    want, slack, *_ = ref.following(x, 2)
    ref.check(h, want, slack)
    ref.check_codes(codes, scales, h)


def vector(shape, seed, scale=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale


def some_cancel(tokens, d, seed):
    """Random rows; of five, one lies far from zero with next to no spread, so that its sums cancel."""
    x = rows((tokens, d), seed)
    far = torch.arange(tokens) % 5 == 2
    g = torch.Generator().manual_seed(seed)
    x[far] = (256.0 + 2.0 * (torch.rand((int(far.sum()), d), generator=g) < 0.02)).to(torch.bfloat16)
    x[far, -1] = 258.0
    return x


@pytest.mark.parametrize("tokens,d", FORMS)
def test_some_rows_of_a_wave_cancel(tokens, d):
    x, y = some_cancel(tokens, d, 1), some_cancel(tokens + 2, d, 2)[2:]
    run_and_check(x, y, post=kq.KQ_NORM_LAYER, pre=kq.KQ_NORM_LAYER, scale=0.5)
    run_and_check(torch.zeros_like(x), y, pre=kq.KQ_NORM_LAYER, eps=1e-3)


@pytest.mark.parametrize("post,pre", [(0, 1), (1, 2), (2, 0), (2, 1), (0, 2)])
@pytest.mark.parametrize("tokens,d", FORMS)
def test_rows_that_are_not_finite_beside_others(tokens, d, post, pre):
    """A NaN or an infinity makes of its row what the formula does, and leaves the rows of the same wave alone."""
    x, y = rows((tokens, d), 1), rows((tokens, d), 2)
    at = torch.arange(tokens)
    x[at % 9 == 1, 3], y[at % 9 == 3, d - 1] = float("nan"), float("inf")
    y[at % 9 == 4, 9], x[at % 9 == 7, d - 2] = float("nan"), -float("inf")
    xs = x.to(DEV)
    out, h, (codes, scales) = torch.empty_like(xs), torch.empty_like(xs), kq.alloc_outputs(xs)
    stats = torch.empty((tokens, 2), device=DEV) if pre else None
    kq.kq_residual_norm(xs, y.to(DEV), out, post=post, pre=pre, h=h, out_codes=codes, out_scales=scales, row_stats=stats)
    ref.check(out, *ref.residual(x, y, post), what="x")
    want, slack, mean, rstd = ref.following(out.cpu(), pre)
    ref.check(h, want, slack, what="h")
    fine = torch.isfinite(want).all(1)
    assert torch.equal(fine, ~torch.isin(at % 9, torch.tensor([1, 3, 4, 7])))
    ref.check_codes(codes.cpu()[fine], scales.cpu()[fine], h.cpu()[fine])
    if pre:
        same_stats(stats.cpu()[fine], mean[fine], rstd[fine], out.cpu()[fine])
        got, want = stats.cpu().double()[~fine], torch.cat((mean, rstd), 1)[~fine]
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isinf(got), torch.isinf(want))


@pytest.mark.parametrize("pre", [0, 1, 2])
@pytest.mark.parametrize("tokens,d", FORMS)
def test_the_stream_alone(tokens, d, pre):
    """Without a block's output, with a weight and a modulation."""
    x, per = rows((tokens, d), 3, 2.0), tokens // 2 + 1
    w, scale, shift = vector(d, 1), vector((2, d), 2, 0.3), vector((2, d), 3, 0.3)
    xs = x.to(DEV)
    h, stats, (codes, scales) = torch.empty_like(xs), torch.empty((tokens, 2), device=DEV), kq.alloc_outputs(xs)
    kq.kq_residual_norm(xs, None, None, pre=pre, pre_weight=w.to(DEV), mod_scale=scale.to(DEV), mod_shift=shift.to(DEV),
                        tokens_per_sample=per, h=h, out_codes=codes, out_scales=scales, row_stats=stats if pre else None)
    assert torch.equal(xs.cpu(), x)
    want, slack, mean, rstd = ref.following(x, pre, w, scale, shift, per)
    ref.check(h, want, slack)
    ref.check_codes(codes, scales, h)
    if pre:
        same_stats(stats, mean, rstd, x)


@pytest.mark.parametrize("post,pre", [(0, 0), (1, 0), (2, 1), (1, 2)])
@pytest.mark.parametrize("tokens,d", FORMS)
def test_every_part(tokens, d, post, pre):
    per = tokens // 2 + 1
    run_and_check(rows((tokens, d), 5), rows((tokens, d), 6, 3.0), per=per, post=post, pre=pre, post_weight=vector(d, 1),
                  gate=vector((2, d), 2), scale=0.5, pre_weight=vector(d, 3), mod_scale=vector((2, d), 4),
                  mod_shift=vector((2, d), 5))


@pytest.mark.parametrize("tokens,d", FORMS)
def test_in_place_and_in_columns(tokens, d):
    x, y, gate = rows((tokens, d), 7), rows((tokens, d), 8), vector((1, d), 9)
    run_and_check(x, y, post=1, pre=2, gate=gate, in_place=True)
    wide = torch.empty((tokens, 3 * d + 24), dtype=torch.bfloat16)
    wide[:, :d], wide[:, d:2 * d], wide[:, 2 * d:] = x, y, 7.0
    m = wide.to(DEV)
    kq.kq_residual_norm(m[:, :d], m[:, d:2 * d], m[:, :d], post=1, gate=gate.to(DEV), pre=2, h=m[:, 2 * d + 16:3 * d + 16])
    got = m.cpu()
    ref.check(got[:, :d], *ref.residual(x, y, 1, gate=gate))
    want, slack, *_ = ref.following(got[:, :d], 2)
    ref.check(got[:, 2 * d + 16:3 * d + 16], want, slack)
    assert torch.equal(got[:, d:2 * d], y)
    assert (got[:, 2 * d:2 * d + 16] == 7).all() and (got[:, 3 * d + 16:] == 7).all()


@pytest.mark.parametrize("tokens,d,per", [(7460001, 1152, None), (524291, 16384, 1), (2051, 1 << 20, 1)])
def test_everything_past_4_gib(tokens, d, per):
    """Rows, h and codes (rows to waves and to workgroups) and the vectors of samples of one row (rows to workgroups, rows
    read again) beyond byte 2^32: the last rows are right, the zeros before them give zeros."""
    last = 3
    x = torch.zeros((tokens, d), dtype=torch.bfloat16, device=DEV)
    y = torch.zeros_like(x)
    end, add = rows((last, d), 1), rows((last, d), 2)
    x[-last:], y[-last:] = end.to(DEV), add.to(DEV)
    samples = tokens if per else 1
    gate = torch.ones((samples, d), device=DEV)
    ends = vector((last if per else 1, d), 3, 0.5)
    gate[-len(ends):] = ends.to(DEV)
    h, (codes, scales) = torch.empty_like(x), kq.alloc_outputs(x)
    assert h.numel() * 2 > 1 << 32 and (d > 16384 or codes.numel() > 1 << 32) and (not per or gate.numel() * 4 > 1 << 32)
    kq.kq_residual_norm(x, y, x, post=1, gate=gate, pre=1, mod_scale=gate, tokens_per_sample=per, h=h, out_codes=codes,
                        out_scales=scales)
    stored, got = x[-last:].cpu(), h[-last:].cpu()
    ref.check(stored, *ref.residual(end, add, 1, gate=ends, per=per))
    want, slack, *_ = ref.following(stored, 1, None, ends, None, per)
    ref.check(got, want, slack)
    ref.check_codes(codes[-last:], scales[-last:], got)
    for t in (x, h):
        assert not any(part.any() for part in t[:-last].split(1 << 16))
    # a zero keeps the sign that a factor gives it, and its code too
    ref.check_codes(codes[:1], scales[:1], h[:1])
    for t in (codes, scales):
        assert all((part == t[:1]).all() for part in t[:-last].split(1 << 16))
    del x, y, h, gate, codes, scales
    torch.cuda.empty_cache()
