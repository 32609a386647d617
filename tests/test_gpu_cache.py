"""The MXFP4 key/value cache on an MI355X (through the C ABI): rows quantized into their slots equal the oracle's
plain MXFP4 bit for bit, slots read back are exactly the values of their codes, and nothing else is touched."""
import pytest
import torch

import cache_reference as ref

kq = pytest.importorskip("w4a4_diffusion_transformer_amd")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    kq.lib()


def filled(n_slots, width, byte=0xFF):
    return tuple(torch.full((n_slots, w), byte, dtype=torch.uint8, device=DEV)
                 for w in (width // 2, width // 32, width // 2, width // 32))


@pytest.mark.parametrize("tokens,width,n_slots", [(1, 32, 1), (3, 96, 9), (8, 1024, 64), (77, 1152, 200), (513, 2240, 600),
                                                  (2049, 160, 3000), (5, 12288, 7)])
def test_write_and_read(tokens, width, n_slots):
    kv = ref.bf16((tokens, 2 * width), tokens + width, 3.0)
    kv[0, :32] = 0                      # a block of zeros: scale byte 0
    kv[-1, width:width + 32] = 2.0 ** -126
    g = torch.Generator().manual_seed(tokens)
    slots = torch.randperm(n_slots, generator=g)[:tokens].to(torch.int32)
    if tokens > 2:  # tokens without a slot: padding, and past either end
        slots[1], slots[2] = -1, n_slots
    if tokens > 4:
        slots[3], slots[4] = -2 ** 31, 2 ** 31 - 1
    cache = filled(n_slots, width)
    x = kv.to(DEV)
    assert kq.kq_cache_write(x[:, :width], x[:, width:], slots.to(DEV), *cache) == cache  # columns of one matrix
    torch.cuda.synchronize()
    there = (slots >= 0) & (slots < n_slots)
    at = slots[there].long()
    for t, (codes, scales) in zip((kv[:, :width], kv[:, width:]), (cache[:2], cache[2:])):
        want_c, want_s = ref.quantize(t)
        codes, scales = codes.cpu(), scales.cpu()
        assert torch.equal(codes[at], want_c[there]) and torch.equal(scales[at], want_s[there])
        rest = torch.ones(n_slots, dtype=torch.bool)
        rest[at] = False
        assert (codes[rest] == 0xFF).all() and (scales[rest] == 0xFF).all()  # other slots as they were
    # read back: into columns of one matrix, with slots that repeat
    again = torch.cat((slots, slots[:3]))
    n = again.numel()
    out = torch.full((n + 2, 2 * width + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    kq.kq_cache_read(*cache, again.to(DEV), out[:n, :width], out[:n, width:2 * width])
    torch.cuda.synchronize()
    out = out.cpu()
    assert (out[n:] == 7).all() and (out[:, 2 * width:] == 7).all()
    ok = (again >= 0) & (again < n_slots)
    for got, (codes, scales) in zip((out[:n, :width], out[:n, width:2 * width]), (cache[:2], cache[2:])):
        want = ref.values(codes.cpu()[again[ok].long()], scales.cpu()[again[ok].long()])
        assert torch.equal(got[ok].double(), want)
        assert (got[~ok] == 0).all()


def test_keys_alone_and_every_scale():
    codes = torch.arange(16, dtype=torch.uint8).repeat(253, 1) * 17  # both nibbles: every code
    scales = torch.arange(253, dtype=torch.uint8)[:, None]
    out = torch.empty((253, 32), dtype=torch.bfloat16, device=DEV)
    kq.kq_cache_read(codes.to(DEV), scales.contiguous().to(DEV), None, None,
                     torch.arange(253, dtype=torch.int32, device=DEV), out, None)
    assert torch.equal(out.cpu().double(), ref.values(codes, scales))
    # and written without values
    x = ref.bf16((6, 64), 5)
    kc, ks, vc, vs = filled(6, 64)
    kq.kq_cache_write(x.to(DEV), None, torch.arange(6, dtype=torch.int32, device=DEV), kc, ks, None, None)
    want = ref.quantize(x)
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(ks.cpu(), want[1])


def test_pools_past_4_gib():
    """Slots whose codes start beyond byte 2^32: 2.2e6 slots of 4096 channels, 4.5 GB of codes each."""
    width, n = 4096, 2_200_000
    cache = tuple(torch.empty((n, w), dtype=torch.uint8, device=DEV) for w in (2048, 128, 2048, 128))
    slots = torch.tensor([0, 1, 1_048_575, 1_048_576, 2_097_151, 2_097_152, 2_097_153, n - 1], dtype=torch.int32)
    k, v = ref.bf16((8, width), 1), ref.bf16((8, width), 2)
    kq.kq_cache_write(k.to(DEV), v.to(DEV), slots.to(DEV), *cache)
    ko, vo = torch.empty_like(k, device=DEV), torch.empty_like(v, device=DEV)
    kq.kq_cache_read(*cache, slots.to(DEV), ko, vo)
    for x, codes, scales, o in ((k, *cache[:2], ko), (v, *cache[2:], vo)):
        want = ref.quantize(x)
        assert torch.equal(codes[slots.long().to(DEV)].cpu(), want[0])
        assert torch.equal(scales[slots.long().to(DEV)].cpu(), want[1])
        assert torch.equal(o.cpu().double(), ref.values(*want))


def test_no_tokens_and_no_slots():
    cache = filled(4, 64)
    none = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    kq.kq_cache_write(none, none, torch.empty(0, dtype=torch.int32, device=DEV), *cache)
    x = ref.bf16((3, 64), 1).to(DEV)
    at = torch.zeros(3, dtype=torch.int32, device=DEV)
    empty = tuple(torch.empty((0, w), dtype=torch.uint8, device=DEV) for w in (32, 2, 32, 2))
    with pytest.raises(kq.KQError):  # an empty tensor has no address
        kq.kq_cache_write(x, x, at, *empty)
    torch.cuda.synchronize()
    assert all((t == 0xFF).all() for t in cache)


@pytest.mark.parametrize("width", [32, 1152])
def test_read_into_columns_with_the_values_first(width):
    """One matrix whose first columns take V and whose last take K."""
    cache = filled(9, width)
    kv = ref.bf16((9, 2 * width), width)
    at = torch.arange(9, dtype=torch.int32, device=DEV)
    kq.kq_cache_write(kv[:, :width].contiguous().to(DEV), kv[:, width:].contiguous().to(DEV), at, *cache)
    out = torch.full((9, 2 * width + 40), 7.0, dtype=torch.bfloat16, device=DEV)
    kq.kq_cache_read(*cache, at, out[:, width + 40:], out[:, :width])
    got = out.cpu()
    assert torch.equal(got[:, width + 40:].double(), ref.values(*cache[:2]))
    assert torch.equal(got[:, :width].double(), ref.values(*cache[2:]))
    assert (got[:, width:width + 40] == 7).all()
