"""The residual stream between two blocks on an MI355X (through the C ABI), against 64-bit forms: the stream, the next
block's input as rows and as MXFP4, and the statistics that the quantizer reads."""
import pytest
import torch

import block_reference as ref
import cache_reference as cref

kq = pytest.importorskip("w4a4_diffusion_transformer_amd")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    kq.lib()


def gpu(t):
    return None if t is None else t.to(DEV)


def vector(shape, seed, scale=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale


def same_stats(got, mean, rstd, rows):
    """fp32 statistics: one rounding (2^-24) of sums whose fp64 error is below 2^-40 of the terms' sizes."""
    got = got.cpu().double()
    size = rows.double().abs().mean(1)
    assert ((got[:, 0] - mean[:, 0]).abs() <= 2.0 ** -24 * mean[:, 0].abs() + 2.0 ** -40 * size).all()
    assert ((got[:, 1] / rstd[:, 0] - 1).abs() <= 2.0 ** -24 + 2.0 ** -36).all()


def run_and_check(x, y, per=None, post=0, pre=0, post_weight=None, gate=None, scale=1.0, pre_weight=None, mod_scale=None,
                  mod_shift=None, eps=1e-6, in_place=False):
    tokens, d = x.shape
    e = lambda *s: torch.full(s, 7.0, dtype=torch.bfloat16, device=DEV)
    xs = x.to(DEV)
    out, h = (xs if in_place else e(tokens + 1, d)[:tokens]), e(tokens + 1, d)
    codes, scales = kq.alloc_outputs(xs)
    stats = torch.empty((tokens, 2), device=DEV) if pre else None
    kw = dict(post=post, post_weight=gpu(post_weight), gate=gpu(gate), residual_scale=scale, pre=pre,
              pre_weight=gpu(pre_weight), mod_scale=gpu(mod_scale), mod_shift=gpu(mod_shift), tokens_per_sample=per, eps=eps)
    got = kq.kq_residual_norm(xs, y.to(DEV), out, h=h[:tokens], out_codes=codes, out_scales=scales, row_stats=stats, **kw)
    assert got[0] is out
    torch.cuda.synchronize()
    assert (h[tokens:] == 7).all()
    ref.check(out, *ref.residual(x, y, post, post_weight, gate, scale, per, eps), what="x")
    stored = out.cpu()
    want, slack, mean, rstd = ref.following(stored, pre, pre_weight, mod_scale, mod_shift, per, eps)
    ref.check(h[:tokens], want, slack, what="h")
    ref.check_codes(codes, scales, h[:tokens])
    if pre:
        same_stats(stats, mean, rstd, stored)
    if not in_place:  # each output alone is the same
        for which in ("h", "codes", "stats") if pre else ("h", "codes"):
            out2, h2, c2, s2 = e(tokens, d), e(tokens, d), *kq.alloc_outputs(xs)
            st2 = torch.empty((tokens, 2), device=DEV)
            kq.kq_residual_norm(xs, y.to(DEV), out2, h=h2 if which == "h" else None,
                                out_codes=c2 if which == "codes" else None, out_scales=s2 if which == "codes" else None,
                                row_stats=st2 if which == "stats" else None, **kw)
            assert torch.equal(out2, out)
            assert which != "h" or torch.equal(h2, h[:tokens])
            assert which != "codes" or (torch.equal(c2, codes) and torch.equal(s2, scales))
            assert which != "stats" or torch.equal(st2, stats)
        out3 = e(tokens, d)
        kq.kq_residual_norm(xs, y.to(DEV), out3, **kw)  # the stream alone
        assert torch.equal(out3, out)


WIDTHS = [32, 64, 96, 480, 512, 544, 1024, 1152, 1536, 1568, 2240, 2560, 2592, 4096, 5600, 6144, 6176, 12288, 16384, 16416, 20480]


@pytest.mark.parametrize("d", WIDTHS)
def test_widths(d):
    tokens = 13
    run_and_check(cref.bf16((tokens, d), d, 2.0), cref.bf16((tokens, d), d + 1), per=5, post=kq.KQ_NORM_RMS,
                  pre=kq.KQ_NORM_LAYER, post_weight=vector(d, 1), gate=vector((3, d), 2), pre_weight=vector(d, 3),
                  mod_scale=vector((3, d), 4, 0.3), mod_shift=vector((3, d), 5, 0.3))


@pytest.mark.parametrize("post", [0, 1, 2])
@pytest.mark.parametrize("pre", [0, 1, 2])
@pytest.mark.parametrize("parts", ["none", "weights", "gate", "modulation", "scale", "shift", "all"])
def test_parts(post, pre, parts):
    for tokens, d in ((1, 160), (37, 1152)):
        per, every = max(1, tokens // 3), parts == "all"
        n = -(-tokens // per)
        on = lambda name, shape, seed: vector(shape, seed) if every or parts == name else None
        run_and_check(cref.bf16((tokens, d), 1), cref.bf16((tokens, d), 2, 2.0), per=per, post=post, pre=pre,
                      post_weight=on("weights", d, 3), pre_weight=on("weights", d, 4), gate=on("gate", (n, d), 5),
                      mod_scale=vector((n, d), 6) if every or parts in ("modulation", "scale") else None,
                      mod_shift=vector((n, d), 7) if every or parts in ("modulation", "shift") else None,
                      scale=0.7 if every else 1.0)


@pytest.mark.parametrize("tokens,d", [(1, 2240), (9, 1152), (5, 12288), (3, 20480)])
def test_in_place(tokens, d):
    run_and_check(cref.bf16((tokens, d), 1), cref.bf16((tokens, d), 2), post=1, pre=1, gate=vector((1, d), 3), in_place=True)


@pytest.mark.parametrize("tokens", [1, 2, 3, 255, 4099, 33001])
def test_rows(tokens):
    """More rows than the GPU holds at once, and samples that end anywhere."""
    d = 64
    per = max(1, tokens // 3 - 1)
    n = -(-tokens // per)
    run_and_check(cref.bf16((tokens, d), 1), cref.bf16((tokens, d), 2), per=per, post=2, pre=1, gate=vector((n, d), 3),
                  mod_scale=vector((n, d), 4))


@pytest.mark.parametrize("d", [1152, 6144, 20480])
def test_norm_of_the_stream_alone(d):
    """Without a block's output: as kq_row_stats, and as the modulation in 64 bits."""
    tokens = 21
    x = cref.bf16((tokens, d), 4, 2.0)
    e = lambda: torch.empty((tokens, d), dtype=torch.bfloat16, device=DEV)
    scale, shift = vector((2, d), 1, 0.3), vector((2, d), 2, 0.3)
    for pre in (0, 1, 2):
        h, stats, (codes, scales) = e(), torch.empty((tokens, 2), device=DEV), kq.alloc_outputs(x.to(DEV))
        kq.kq_residual_norm(x.to(DEV), None, None, pre=pre, mod_scale=gpu(scale), mod_shift=gpu(shift), tokens_per_sample=11,
                            h=h, out_codes=codes, out_scales=scales, row_stats=stats if pre else None)
        want, slack, mean, rstd = ref.following(x, pre, None, scale, shift, 11)
        ref.check(h, want, slack)
        ref.check_codes(codes, scales, h)
        if pre:
            same_stats(stats, mean, rstd, x)


def test_statistics_feed_the_quantizer():
    """Stream and statistics from one call, codes from kq_quantize_adaln: those of the two-call form."""
    tokens, d, per = 96, 1152, 32
    x, y = cref.bf16((tokens, d), 1).to(DEV), cref.bf16((tokens, d), 2).to(DEV)
    gate, scale, shift = (vector((3, d), s, 0.3).to(DEV) for s in (3, 4, 5))
    g = torch.Generator().manual_seed(6)
    params = torch.randn((d // 32, 5, 3), generator=g)
    params[..., 1] = 1 + 0.2 * params[..., 1].clamp(-2, 2)
    params = params.to(DEV)
    out, stats = torch.empty_like(x), torch.empty((tokens, 2), device=DEV)
    kq.kq_residual_norm(x, y, out, gate=gate, tokens_per_sample=per, pre=kq.KQ_NORM_LAYER, row_stats=stats)
    a = kq.kq_quantize_adaln(out, stats, scale, shift, per, params, *kq.alloc_outputs(x))
    again = kq.kq_row_stats(out, 1e-6, torch.empty_like(stats))
    torch.cuda.synchronize()
    # the two sum in different orders: an fp32 step at most, where a sum lies next to a tie
    assert ((again - stats).abs() <= 2.0 ** -23 * stats.abs()).all()
    b = kq.kq_quantize_adaln(out, again, scale, shift, per, params, *kq.alloc_outputs(x))
    equal = (again == stats).all(1)
    assert equal.float().mean() > 0.9
    assert torch.equal(a[0][equal], b[0][equal]) and torch.equal(a[1][equal], b[1][equal])


def test_a_mean_far_above_the_spread():
    """Rows whose sums of squares cancel: 1 / deviation from a second pass."""
    for d in (1152, 6144, 20480):
        x = torch.full((3, d), 256.0, dtype=torch.bfloat16)
        x[0, 5], x[1, 7:90] = 258.0, 254.0
        y = torch.zeros_like(x)
        y2 = x.clone()
        run_and_check(x, y, post=0, pre=2)
        run_and_check(y, y2, post=2, pre=2, eps=1e-3)


def test_rows_of_one_value_and_of_zeros():
    d = 96
    x = torch.zeros((3, d), dtype=torch.bfloat16)
    x[1] = 5.0
    run_and_check(x, torch.zeros_like(x), post=1, pre=2)
    run_and_check(x, x, post=2, pre=1)


def test_values_that_are_not_finite():
    """A row with a NaN or an infinity gives what the formula gives; other rows are not touched."""
    for d in (64, 6144):
        x, y = cref.bf16((5, d), 1), cref.bf16((5, d), 2)
        x[1, 3], y[2, 9], y[3, 33], x[4, 8] = float("nan"), float("inf"), float("nan"), -float("inf")
        for post in (0, 1):
            out, h = (torch.empty((5, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
            kq.kq_residual_norm(x.to(DEV), y.to(DEV), out, post=post, pre=1, h=h)
            ref.check(out, *ref.residual(x, y, post), what=f"x {post}")
            want, slack, *_ = ref.following(out.cpu(), 1)
            ref.check(h, want, slack, what=f"h {post}")


def test_columns_of_wider_matrices():
    tokens, d = 11, 96
    wide = cref.bf16((tokens, 4 * d + 8), 3)
    m = wide.to(DEV)
    x, y, out, h = m[:, :d], m[:, d:2 * d], m[:, 2 * d:3 * d], m[:, 3 * d + 8:]
    kq.kq_residual_norm(x, y, out, post=1, pre=1, h=h)
    got = m.cpu()
    assert torch.equal(got[:, :2 * d], wide[:, :2 * d]) and torch.equal(got[:, 3 * d:3 * d + 8], wide[:, 3 * d:3 * d + 8])
    ref.check(got[:, 2 * d:3 * d], *ref.residual(wide[:, :d], wide[:, d:2 * d], 1))
    want, slack, *_ = ref.following(got[:, 2 * d:3 * d], 1)
    ref.check(got[:, 3 * d + 8:], want, slack)


def test_rows_past_4_gib():
    """Rows, codes and vectors beyond byte 2^32, samples of one row."""
    tokens, d = 1100, 1 << 21
    x = torch.zeros((tokens, d), dtype=torch.bfloat16, device=DEV)
    last = cref.bf16((2, d), 5)
    x[-2:] = last.to(DEV)
    codes, scales = kq.alloc_outputs(x)
    stats = torch.empty((tokens, 2), device=DEV)
    kq.kq_residual_norm(x, x.clone(), x, residual_scale=0.5, pre=1, out_codes=codes, out_scales=scales, row_stats=stats)
    stored = x[-2:].cpu()
    ref.check(stored, *ref.residual(last, last, scale=0.5))
    want, slack, mean, rstd = ref.following(stored, 1)
    same_stats(stats[-2:], mean, rstd, stored)
    rows = ref.rounded(want)
    sure = (ref.between(want, slack)[0] == ref.between(want, slack)[1]).all()
    if sure:
        ref.check_codes(codes[-2:], scales[-2:], rows.to(torch.bfloat16))
    assert not codes[:-2].any() and not scales[:-2].any()


@pytest.mark.parametrize("d", [64, 1152])
def test_rows_far_apart(d):
    """Strides at which a wave takes one row."""
    tokens, stride = 7300 if d == 64 else 1900, (1 << 20) + 8
    flat = torch.empty((tokens - 1) * stride + d, dtype=torch.bfloat16, device=DEV)
    far = flat.as_strided((tokens, d), (stride, 1))
    x, y = cref.bf16((tokens, d), 1), cref.bf16((tokens, d), 2)
    far.copy_(x.to(DEV))
    gate = vector((1, d), 3)
    for out in (far, torch.empty((tokens, d), dtype=torch.bfloat16, device=DEV)):
        far.copy_(x.to(DEV))
        codes, scales = kq.alloc_outputs(y)
        codes, scales = codes.to(DEV), scales.to(DEV)
        kq.kq_residual_norm(far, y.to(DEV), out, post=1, pre=1, gate=gate.to(DEV), out_codes=codes, out_scales=scales)
        stored = out.cpu()
        ref.check(stored, *ref.residual(x, y, 1, gate=gate))
        want, slack, *_ = ref.following(stored, 1)
        lo, hi = ref.between(want, slack)
        same = (lo == hi).view(tokens, -1, 32).all(2).all(1)  # rows without a tie
        assert same.float().mean() > 0.99
        ref.check_codes(codes.cpu()[same], scales.cpu()[same], lo[same].to(torch.bfloat16))
    del flat, far


# pieces a lane and rows a wave: the choices of the launch at many rows
@pytest.mark.parametrize("tokens,d", [(33001, 32), (17003, 96), (9101, 160), (18001, 256), (33000, 128), (7301, 512), (17001, 512),
                                      (3701, 736), (16385, 736), (7199, 800), (1801, 1152), (9001, 1152), (2801, 1536),
                                      (4100, 1760), (2051, 2240), (1100, 2592), (1100, 3040)])
def test_many_rows(tokens, d):
    g = torch.Generator().manual_seed(d)
    x = (torch.randn((tokens, d), generator=g)).to(torch.bfloat16)
    y = (torch.randn((tokens, d), generator=g) * 2).to(torch.bfloat16)
    per = tokens // 3 + 1
    run_and_check(x, y, per=per, post=1, pre=2, post_weight=vector(d, 1), gate=vector((3, d), 2), mod_shift=vector((3, d), 3))


def test_no_rows():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    kq.kq_residual_norm(x, x, x, pre=1, h=x)
    torch.cuda.synchronize()
