"""Edges of the residual stream's norms on an MI355X (through the C ABI): sums that cancel, values that are not finite and
missing parts, at the row counts and widths that take each of the kernel's forms, with such rows beside others."""
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
