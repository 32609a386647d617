"""kq_gemm_mx_ex on an MI355X: the W4A4 product with bias, activation, gate and residual against 64 bits."""
import numpy as np
import pytest
import torch

import cache_reference as ref

kq = pytest.importorskip("w4a4_diffusion_transformer_amd")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ACTS = {"none": 0, "gelu_tanh": 1, "gelu_erf": 2, "silu": 3}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    kq.lib()


def operands(m, n, k, seed):
    rng = np.random.default_rng(seed)
    t = lambda r, w, lo, hi: torch.from_numpy(rng.integers(lo, hi, size=(r, w), dtype=np.uint8))
    return t(m, k // 2, 0, 256), t(m, k // 32, 122, 128), t(n, k // 2, 0, 256), t(n, k // 32, 120, 126)


def extras(m, n, rps, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, generator=g), torch.randn((-(-m // rps), n), generator=g),
            torch.randn((m, n), generator=g).to(torch.bfloat16))


def run(ops, bias, name, gate, rps, residual, fp32=True, bf16=True, in_place=False):
    d = lambda t: None if t is None else t.to(DEV)
    m, n = ops[0].shape[0], ops[2].shape[0]
    y = torch.full((m, n), 7.0, device=DEV) if fp32 else None
    res = d(residual)
    yb = res if in_place else torch.full((m, n), 7.0, dtype=torch.bfloat16, device=DEV) if bf16 else None
    kq.kq_gemm_mx_ex(*map(d, ops), bias=d(bias), act=ACTS[name], gate=d(gate), rows_per_sample=rps, residual=res,
                     y_f32=y, y_bf16=yb)
    torch.cuda.synchronize()
    return y, yb


SIZES = [(1, 1, 32), (1, 6912, 1152), (2, 100, 5600), (7, 33, 96), (16, 640, 2240), (17, 257, 160), (32, 64, 12288),
         (33, 130, 1504), (64, 1152, 1152), (100, 300, 320), (129, 45, 64), (300, 257, 2240), (512, 384, 1152),
         (1000, 520, 96),
         # past the few-row form: half tiles, rows of any alignment, 192-row tiles, whole tiles and halves
         (1400, 1000, 96), (1201, 1101, 160), (2500, 600, 2240), (3333, 2600, 96), (3333, 2601, 1504), (4352, 4096, 128)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_everything_at_every_size(m, n, k):
    ops = operands(m, n, k, m + n + k)
    rps = max(1, m // 3)
    bias, gate, residual = extras(m, n, rps, m)
    want, tol = ref.gemm(*ops, bias, "gelu_tanh", gate, rps, residual)
    y, yb = run(ops, bias, "gelu_tanh", gate, rps, residual)
    assert ((y.cpu().double() - want).abs() <= tol).all()
    assert torch.equal(yb, y.to(torch.bfloat16))  # the same value, rounded once


@pytest.mark.parametrize("m,n,k", [(3, 70, 96), (40, 70, 96), (300, 70, 96), (1300, 1040, 64)])
@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("parts", ["", "b", "g", "r", "bg", "gr", "br"])
def test_each_part_alone(m, n, k, name, parts):
    ops = operands(m, n, k, 3)
    rps = 7 if m < 1000 else 500
    bias, gate, residual = extras(m, n, rps, 4)
    bias, gate, residual = bias if "b" in parts else None, gate if "g" in parts else None, residual if "r" in parts else None
    want, tol = ref.gemm(*ops, bias, name, gate, rps, residual)
    y, yb = run(ops, bias, name, gate, rps, residual)
    assert ((y.cpu().double() - want).abs() <= tol).all()
    assert torch.equal(yb, y.to(torch.bfloat16))


@pytest.mark.parametrize("m", [1, 20, 48, 300, 9001])
def test_residual_in_place(m):
    ops = operands(m, 150, 128, 5)
    bias, gate, residual = extras(m, 150, m, 6)
    _, apart = run(ops, bias, "none", gate, None, residual, fp32=False)
    _, same = run(ops, bias, "none", gate, None, residual, fp32=False, in_place=True)
    assert torch.equal(apart, same)


@pytest.mark.parametrize("m", [2, 30, 260, 21000])
def test_activation_tails(m):
    """Biases that reach far into both tails of each activation; results stay finite and exact to the bound."""
    ops = operands(m, 64, 32, 9)
    bias = torch.linspace(-200, 200, 64)
    for name in ACTS:
        want, tol = ref.gemm(*ops, bias, name, None, 1, None)
        y, _ = run(ops, bias, name, None, 1, None)
        assert torch.isfinite(y).all() and ((y.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("m,n", [(2, 3), (5, 300), (70, 2), (300, 257)])
def test_plain_product_of_one_block(m, n):
    """kq_gemm_mx at K = 32: every row has one scale byte, also the last rows, whose neighbours end the tensor."""
    ops = operands(m, n, 32, 11)
    want, tol = ref.gemm(*ops, None, "none", None, 1, None)
    y = torch.empty((m, n), device=DEV)
    kq.kq_gemm_mx(*[t.to(DEV) for t in ops], y_f32=y)
    assert ((y.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("m,n", [(1, 1), (257, 258), (258, 513), (1030, 1281), (1, 2000), (1400, 3)])
def test_one_block_whose_last_rows_are_in_two_tiles(m, n):
    """The same with the last three rows on both sides of a tile's end, and fewer rows than three."""
    ops = operands(m, n, 32, 12)
    want, tol = ref.gemm(*ops, None, "none", None, 1, None)
    y, z = torch.empty((2, m, n), device=DEV)
    ops = [t.to(DEV) for t in ops]
    kq.kq_gemm_mx(*ops, y_f32=y)
    kq.kq_gemm_mx_ex(*ops, y_f32=z)
    assert ((y.cpu().double() - want).abs() <= tol).all() and ((z.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("m,n", [(1100, 1300), (3333, 2600)])
def test_same_sums_as_the_plain_product(m, n):
    """Above the sizes of the few-row form, without any part, the bits are kq_gemm_mx's."""
    ops = [t.to(DEV) for t in operands(m, n, 2240, 10)]
    a, b = (torch.empty((m, n), device=DEV) for _ in range(2))
    kq.kq_gemm_mx(*ops, y_f32=a)
    kq.kq_gemm_mx_ex(*ops, y_f32=b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("m,n", [(40, 72), (1400, 1000)])
def test_outputs_and_residuals_that_start_anywhere(m, n):
    """Rows of a whole number of 16-byte pieces whose matrices do not start at one: element accesses."""
    ops = operands(m, n, 64, 12)
    bias, gate, residual = extras(m, n, m, 13)
    want, tol = ref.gemm(*ops, bias, "silu", gate, m, residual)
    res = torch.empty(m * n + 1, dtype=torch.bfloat16, device=DEV)[1:].view(m, n)
    res.copy_(residual)
    flat = torch.full((m * n + 2,), 7.0, device=DEV)
    y = flat[1:-1].view(m, n)
    kq.kq_gemm_mx_ex(*[t.to(DEV) for t in ops], bias=bias.to(DEV), act=ACTS["silu"], gate=gate.to(DEV), residual=res, y_f32=y)
    assert ((y.cpu().double() - want).abs() <= tol).all()
    assert flat[0] == 7 and flat[-1] == 7


# half tiles; 192-row tiles; whole tiles and halves; whole tiles of more rows than 192-row ones fit the GPU
TILES = [(1100, 1300, 64), (3333, 2600, 96), (4352, 4096, 32), (5111, 2568, 512)]


@pytest.mark.parametrize("m,n,k", TILES)
def test_every_row_and_channel_of_a_tile(m, n, k):
    """The sums reach the epilogue through local memory, each wave's through a part of its own: with a bias the bits are
    the plain product's, which stores from registers, and one fp32 addition's."""
    ops = [t.to(DEV) for t in operands(m, n, k, 14)]
    bias = torch.randn(n, generator=torch.Generator().manual_seed(15)).to(DEV)
    a = torch.empty((m, n), device=DEV)
    y = torch.full((m, n), 7.0, device=DEV)
    yb = torch.full((m, n), 7.0, dtype=torch.bfloat16, device=DEV)
    kq.kq_gemm_mx(*ops, y_f32=a)
    kq.kq_gemm_mx_ex(*ops, bias=bias, y_f32=y, y_bf16=yb)
    assert torch.equal(y, a + bias) and torch.equal(yb, (a + bias).to(torch.bfloat16))


@pytest.mark.parametrize("m,n,k", TILES)
def test_bands_of_a_wave_follow_one_another(m, n, k):
    """Every part of the epilogue, in place: each band of rows is read from local memory whole before the next one
    takes its place.  Each part is one fp32 operation on the plain product, so the bits are torch's."""
    ops = [t.to(DEV) for t in operands(m, n, k, 16)]
    rps = m // 3
    bias, gate, residual = (t.to(DEV) for t in extras(m, n, rps, 17))
    a = torch.empty((m, n), device=DEV)
    kq.kq_gemm_mx(*ops, y_f32=a)
    want = (residual.float() + (a + bias) * gate.repeat_interleave(rps, 0)[:m]).to(torch.bfloat16)
    for _ in range(3):
        x = residual.clone()
        kq.kq_gemm_mx_ex(*ops, bias=bias, gate=gate, rows_per_sample=rps, residual=x, y_bf16=x)
        assert torch.equal(x, want)
