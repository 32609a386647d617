"""Rotary positions and the rotated cache append on an MI355X (through the C ABI), against 64-bit forms; keys in the
cache equal the codes of the rows that kq_rope gives, bit for bit."""
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


def turn(tokens, dims, halves, seed, far=300, base=10000.0):
    """A rotation on the CPU: (positions, freqs, dims, halves)."""
    g = torch.Generator().manual_seed(seed)
    positions = torch.randint(-far, far + 1, (tokens, len(dims)), generator=g, dtype=torch.int64).to(torch.int32)
    return positions, kq.rope_freqs(dims, base, "cpu"), tuple(dims), halves


def on_gpu(rotation):
    return None if rotation is None else kq.Rotation(rotation[0].to(DEV), rotation[1].to(DEV), *rotation[2:])


def weights(dim, seed):
    return torch.rand(dim, generator=torch.Generator().manual_seed(seed)) + 0.5


# tokens, heads, dim, axes, halves, norm
SHAPES = [(1, 1, 8, (8,), False, True), (1, 32, 128, (128,), True, True), (7, 3, 24, (8, 8, 8), False, True),
          (33, 16, 72, (36, 36), False, False), (33, 16, 72, (36, 36), False, True), (5, 4, 72, (72,), True, True),
          (65, 5, 40, (20, 20), True, True), (19, 2, 104, (52, 20, 32), True, False), (130, 20, 96, (64,), True, False),
          (130, 20, 96, (16, 24, 24), False, True), (3, 7, 120, (60, 30, 28, 2), False, True), (11, 8, 64, (6,), True, True),
          (9, 8, 64, (6,), False, True), (257, 6, 128, (16, 56, 56), False, True), (64, 1, 16, (16,), True, True),
          (4097, 2, 64, (64,), False, True), (12, 3, 88, (), False, True), (6, 4, 32, (), False, False),
          (50, 9, 56, (2, 2, 2, 2), True, True), (21, 40, 112, (112,), True, True)]


@pytest.mark.parametrize("tokens,heads,dim,axes,halves,norm", SHAPES)
def test_rope(tokens, heads, dim, axes, halves, norm):
    x = cref.bf16((tokens, heads * dim), tokens + dim, 3.0)
    x[0, :dim] = 0
    rotation = turn(tokens, axes, halves, heads) if axes else None
    for w in (weights(dim, 5), None):
        want = ref.rope(x, heads, rotation, norm, w)
        out = torch.full((tokens + 1, heads * dim), 7.0, dtype=torch.bfloat16, device=DEV)
        assert kq.kq_rope(x.to(DEV), out[:tokens], heads, on_gpu(rotation), kq.KQ_NORM_RMS if norm else kq.KQ_NORM_NONE,
                          None if w is None else w.to(DEV)) is not None
        ref.check(out[:tokens], *want)
        assert (out[tokens:] == 7).all()
        if not norm:
            break


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("dim,axes", [(128, (128,)), (72, (24, 24))])
def test_rope_in_place_and_in_columns(halves, dim, axes):
    """In columns of a wider matrix, then into columns next to them, then in place."""
    tokens, heads, W = 37, 4, 4 * dim
    full = cref.bf16((tokens, 3 * W + 8), 3)
    rotation = turn(tokens, axes, halves, 1)
    want = ref.rope(full[:, W:2 * W], heads, rotation, True, weights(dim, 2))
    args = (heads, on_gpu(rotation), kq.KQ_NORM_RMS, weights(dim, 2).to(DEV))
    x = full.to(DEV)
    kq.kq_rope(x[:, W:2 * W], x[:, 2 * W:3 * W], *args)
    got = x.cpu()
    ref.check(got[:, 2 * W:3 * W], *want)
    assert torch.equal(got[:, :2 * W], full[:, :2 * W]) and torch.equal(got[:, 3 * W:], full[:, 3 * W:])
    kq.kq_rope(x[:, W:2 * W], x[:, W:2 * W], *args)
    assert torch.equal(x[:, W:2 * W].cpu(), got[:, 2 * W:3 * W]) and torch.equal(x[:, :W].cpu(), full[:, :W])


@pytest.mark.parametrize("halves", [False, True])
def test_far_positions(halves):
    """Positions up to the type's ends: an angle is known to 2^-51 of its size, and no worse."""
    tokens = 40
    rotation = list(turn(tokens, (64,), halves, 4))
    ends = torch.tensor([-2 ** 31, 2 ** 31 - 1, -1, 0, 1, 1 << 20, (1 << 24) + 1, -(1 << 28) - 1])
    rotation[0] = ends.repeat(5)[:, None].to(torch.int32).contiguous()
    x = cref.bf16((tokens, 128), 6)
    out = torch.empty_like(x, device=DEV)
    kq.kq_rope(x.to(DEV), out, 2, on_gpu(rotation))
    ref.check(out, *ref.rope(x, 2, rotation))


def test_angles_at_whole_quarters():
    """Angles that are whole multiples of pi / 4, both signs, each octant."""
    tokens = 33
    rotation = (torch.arange(-16, 17, dtype=torch.int32)[:, None], torch.full((4,), torch.pi / 4, dtype=torch.float64), (8,), False)
    x = cref.bf16((tokens, 8), 8)
    out = torch.empty_like(x, device=DEV)
    kq.kq_rope(x.to(DEV), out, 1, on_gpu(rotation))
    ref.check(out, *ref.rope(x, 1, rotation))


@pytest.mark.parametrize("halves", [False, True])
def test_values_that_are_not_finite(halves):
    """Only what the formula makes NaN or infinite: channels that do not turn, other heads and tokens stay."""
    x = cref.bf16((4, 2 * 48), 9)
    x[0, 40], x[1, 3], x[2, 50], x[3, 47] = float("inf"), float("nan"), -float("inf"), float("nan")
    rotation = turn(4, (12, 8), halves, 3)
    for norm in (False, True):
        out = torch.empty_like(x, device=DEV)
        kq.kq_rope(x.to(DEV), out, 2, on_gpu(rotation), kq.KQ_NORM_RMS if norm else kq.KQ_NORM_NONE)
        ref.check(out, *ref.rope(x, 2, rotation, norm), what=f"norm {norm}")


def test_largest_and_smallest_values():
    big = torch.full((2, 64), 3.38e38).to(torch.bfloat16)
    small = torch.full((2, 64), 2.0 ** -126).to(torch.bfloat16)
    rotation = turn(2, (64,), True, 3)
    for x, norm in ((big, True), (small, True), (small, False)):
        out = torch.empty_like(x, device=DEV)
        kq.kq_rope(x.to(DEV), out, 1, on_gpu(rotation), int(norm), eps=0.0)
        want, slack = ref.rope(x, 1, rotation, norm, eps=0.0)
        if not norm:  # below 2^-126 a value may go through one more rounding, of fp32's last step
            slack = slack + 2.0 ** -134
        ref.check(out, want, slack)


# tokens, q_heads (0: none), kv_heads, dim, axes, halves, norm, values
APPENDS = [(1, 32, 8, 128, (128,), True, True, True), (8, 32, 8, 128, (16, 56, 56), False, True, True),
           (33, 0, 16, 72, (36, 36), False, True, True), (29, 4, 4, 72, (72,), True, True, True),
           (77, 10, 10, 80, (40,), True, False, True), (5, 7, 4, 8, (8,), False, True, True),
           (13, 4, 4, 24, (6, 6, 4), True, True, False), (700, 20, 10, 96, (64,), True, False, True),
           (41, 0, 2, 112, (112,), True, True, False), (9, 3, 4, 104, (52, 52), False, True, True),
           (70, 8, 1, 64, (), False, True, True), (3, 6, 2, 16, (16,), False, False, True),
           (1300, 12, 4, 120, (60, 60), True, True, True), (18, 5, 4, 56, (4, 4), False, True, True)]


@pytest.mark.parametrize("tokens,q_heads,kv_heads,dim,axes,halves,norm,values", APPENDS)
def test_append(tokens, q_heads, kv_heads, dim, axes, halves, norm, values):
    q, W = q_heads * dim, kv_heads * dim
    qw = -(-q // 8) * 8
    qkv = cref.bf16((tokens, qw + 2 * W), tokens, 2.0)
    n_slots = tokens + 9
    g = torch.Generator().manual_seed(tokens)
    slots = torch.randperm(n_slots, generator=g)[:tokens].to(torch.int32)
    if tokens > 4:  # tokens without a slot
        slots[1], slots[2], slots[4] = -1, n_slots, -2 ** 31
    rotation = turn(tokens, axes, halves, 3) if axes else None
    kind = kq.KQ_NORM_RMS if norm else kq.KQ_NORM_NONE
    wq, wk = weights(dim, 1), weights(dim, 2)
    x = qkv.to(DEV)
    pools = tuple(torch.full((n_slots, w), 0xAB, dtype=torch.uint8, device=DEV) for w in (W // 2, W // 32) * 2)
    out = torch.full((tokens + 1, q or 8), 7.0, dtype=torch.bfloat16, device=DEV)
    K, V = x[:, qw:qw + W], x[:, qw + W:]
    kq.kq_cache_write_rope(K, V if values else None, slots.to(DEV), *pools, kv_heads, on_gpu(rotation), kind, wk.to(DEV),
                           Q=x[:, :q] if q else None, q_out=out[:tokens] if q else None, q_heads=q_heads,
                           q_weight=wq.to(DEV))
    assert torch.equal(x.cpu(), qkv) and (out[tokens:] == 7).all()
    if q:  # also of tokens without a slot
        ref.check(out[:tokens], *ref.rope(qkv[:, :q], q_heads, rotation, norm, wq), what="q")
    # the same in two steps
    turned = torch.empty((tokens, W), dtype=torch.bfloat16, device=DEV)
    kq.kq_rope(K, turned, kv_heads, on_gpu(rotation), kind, wk.to(DEV))
    ref.check(turned, *ref.rope(qkv[:, qw:qw + W], kv_heads, rotation, norm, wk), what="k")
    two = tuple(torch.full_like(p, 0xAB) for p in pools)
    kq.kq_cache_write(turned, V if values else None, slots.to(DEV), *two)
    for a, b in zip(pools, two):
        assert torch.equal(a, b)
    there = (slots >= 0) & (slots < n_slots)
    at = slots[there].long()
    ref.check_codes(pools[0].cpu()[at], pools[1].cpu()[at], turned.cpu()[there], "keys")
    if values:
        ref.check_codes(pools[2].cpu()[at], pools[3].cpu()[at], qkv[:, qw + W:][there], "values")


def test_append_in_place_in_a_fused_projection():
    """Queries turned in place between the columns of one matrix that keys and values are read from."""
    tokens, heads, kv_heads, dim = 53, 8, 2, 64
    q, W = heads * dim, kv_heads * dim
    qkv = cref.bf16((tokens, q + 2 * W), 8)
    rotation = turn(tokens, (64,), True, 2)
    slots = torch.arange(tokens, dtype=torch.int32, device=DEV)
    for order in ("qkv", "kvq"):
        x = qkv.to(DEV)
        at = 0 if order == "qkv" else 2 * W
        k = q if order == "qkv" else 0
        pools = kq.alloc_cache(tokens, W, DEV)
        kq.kq_cache_write_rope(x[:, k:k + W], x[:, k + W:k + 2 * W], slots, *pools, kv_heads, on_gpu(rotation),
                               Q=x[:, at:at + q], q_out=x[:, at:at + q], q_heads=heads)
        got = x.cpu()
        ref.check(got[:, at:at + q], *ref.rope(qkv[:, at:at + q], heads, rotation))
        assert torch.equal(got[:, k:k + 2 * W], qkv[:, k:k + 2 * W])
        turned = ref.rounded(ref.rope(qkv[:, k:k + W], kv_heads, rotation)[0]).to(torch.bfloat16)
        ref.check_codes(pools[0], pools[1], turned)


def test_append_without_slots_or_tokens():
    x = cref.bf16((3, 64), 1).to(DEV)
    pools = tuple(torch.full((4, w), 0xAB, dtype=torch.uint8, device=DEV) for w in (32, 2, 32, 2))
    none = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    at = torch.full((3,), -1, dtype=torch.int32, device=DEV)
    kq.kq_cache_write_rope(none, none, at[:0], *pools, 1)
    kq.kq_cache_write_rope(x, x, at, *pools, 1)
    kq.kq_rope(none, none, 2)
    torch.cuda.synchronize()
    assert all((p == 0xAB).all() for p in pools)


def test_pools_past_4_gib():
    """Slots whose codes start beyond byte 2^32, heads whose blocks span two."""
    heads, dim = 32, 120
    width, n = heads * dim, 2_400_000
    pools = tuple(torch.empty((n, w), dtype=torch.uint8, device=DEV) for w in (width // 2, width // 32) * 2)
    slots = torch.tensor([0, 2_236_961, 2_236_962, 2_236_963, n - 1], dtype=torch.int32)
    k, v = cref.bf16((5, width), 1), cref.bf16((5, width), 2)
    rotation = turn(5, (120,), False, 3)
    kq.kq_cache_write_rope(k.to(DEV), v.to(DEV), slots.to(DEV), *pools, heads, on_gpu(rotation))
    turned = ref.rounded(ref.rope(k, heads, rotation)[0]).to(torch.bfloat16)
    at = slots.long().to(DEV)
    ref.check_codes(pools[0][at], pools[1][at], turned)
    ref.check_codes(pools[2][at], pools[3][at], v)


def test_rows_past_4_gib():
    """Rows whose elements lie beyond 2^31, at a stride."""
    tokens, stride, heads, dim = 5, 1 << 29, 2, 64
    flat = torch.zeros(4 * stride + 256, dtype=torch.bfloat16, device=DEV)
    x = flat.as_strided((tokens, heads * dim), (stride, 1))
    rows = cref.bf16((tokens, heads * dim), 7)
    x.copy_(rows.to(DEV))
    rotation = turn(tokens, (64,), True, 3)
    kq.kq_rope(x, x, heads, on_gpu(rotation))
    ref.check(x.contiguous(), *ref.rope(rows, heads, rotation))


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("dim,kv_heads", [(128, 3), (64, 5), (72, 4), (16, 2)])
def test_keys_far_apart(dim, kv_heads, halves):
    """Strides that no buffer spans over the tokens of a wave."""
    W, tokens, stride = kv_heads * dim, 5, (1 << 29) + 8
    flat = torch.zeros((tokens - 1) * stride + W, dtype=torch.bfloat16, device=DEV)
    k = flat.as_strided((tokens, W), (stride, 1))
    rows = cref.bf16((tokens, W), 4)
    k.copy_(rows.to(DEV))
    rotation = turn(tokens, (dim,), halves, 3)
    pools = kq.alloc_cache(tokens, W, DEV)
    slots = torch.arange(tokens, dtype=torch.int32, device=DEV)
    kq.kq_cache_write_rope(k, None, slots, pools[0], pools[1], None, None, kv_heads, on_gpu(rotation), kq.KQ_NORM_RMS)
    turned = ref.rounded(ref.rope(rows, kv_heads, rotation, True)[0]).to(torch.bfloat16)
    ref.check_codes(pools[0], pools[1], turned)


def test_more_heads_than_a_round_of_the_gpu():
    """Many tokens of small heads, and one token of many."""
    for tokens, heads, dim in ((70001, 1, 8), (1, 4099, 8), (2, 700, 72)):
        x = cref.bf16((tokens, heads * dim), tokens)
        rotation = turn(tokens, (8,), False, 3)
        out = torch.empty_like(x, device=DEV)
        kq.kq_rope(x.to(DEV), out, heads, on_gpu(rotation), kq.KQ_NORM_RMS)
        ref.check(out, *ref.rope(x, heads, rotation, True))


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("axes", [(6,), (10, 4), (8,), ()])
def test_channels_that_do_not_turn(halves, axes):
    """They come out as they are, the sign of a zero with them; an infinite weight of one makes that one infinite."""
    tokens, heads, dim, R = 5, 3, 64, sum(axes)
    x = cref.bf16((tokens, heads * dim), 5)
    x.view(tokens, heads, dim)[:, :, 20:40:3] = -0.0
    x.view(tokens, heads, dim)[:, :, 21:40:3] = 0.0
    rotation = turn(tokens, axes, halves, 3) if axes else None
    out = torch.empty_like(x, device=DEV)
    kq.kq_rope(x.to(DEV), out, heads, on_gpu(rotation))
    kept = lambda t: t.cpu().view(torch.int16).view(tokens, heads, dim)[:, :, R:]
    assert torch.equal(kept(out), kept(x))
    ref.check(out, *ref.rope(x, heads, rotation))
    w = weights(dim, 4)
    w[41], w[44], w[50] = float("inf"), -float("inf"), -1.0
    kq.kq_rope(x.to(DEV), out, heads, on_gpu(rotation), kq.KQ_NORM_RMS, w.to(DEV))
    want = ref.rope(x, heads, rotation, True, w)
    assert torch.isinf(want[0]).sum() == 2 * tokens * heads
    ref.check(out, *want)
    zero = x.view(tokens, heads, dim)[:, :, 20:40] == 0
    assert torch.equal(torch.signbit(out.cpu().view(tokens, heads, dim)[:, :, 20:40][zero]),
                       torch.signbit(x.view(tokens, heads, dim)[:, :, 20:40][zero]))
