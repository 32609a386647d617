"""Refusals of the rotary, rotated cache-append and residual-norm entry points, without a GPU: the C ABI returns before any
HIP call, the binding raises on tensors that do not fit one another."""
import ctypes
import os

import pytest
import torch

import w4a4_diffusion_transformer_amd as kq

OK, NULL, SHAPE, ALIGN, VARIANT, HIP, ALIAS, WORKSPACE = range(8)
A, B, C, D, E, F, G, H, I, J = (i << 28 for i in range(1, 11))  # aligned fake device addresses
KEPT = []
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kq.LIB_PATH):
        pytest.skip("libkq.so not built")
    return kq.lib()


def turn(dims=(16, 24, 24), positions=I, freqs=J, layout=0, n=None):
    r = kq._CRotation(positions, freqs, len(dims) if n is None else n, (ctypes.c_int32 * 4)(*dims[:4]), layout)
    KEPT.append(r)  # the call reads it
    return ctypes.addressof(r)


def rope(lib, x=A, xs=256, t=4, heads=4, dim=64, norm=1, w=B, eps=1e-6, rotation=None, out=C, os_=256):
    return lib.kq_rope(x, xs, t, heads, dim, norm, w, eps, rotation, out, os_, None)


def test_rope_checks(lib):
    r = lambda **kw: rope(lib, **kw)
    for bad in (dict(t=-1), dict(t=1 << 28), dict(heads=0), dict(heads=-1), dict(heads=(1 << 24) + 1), dict(dim=0),
                dict(dim=60), dict(dim=136), dict(dim=-8), dict(xs=248), dict(xs=260), dict(os_=128), dict(eps=-1.0),
                dict(eps=NAN), dict(eps=INF), dict(rotation=turn((16,), n=5)), dict(heads=1 << 21, dim=128, xs=1 << 28, os_=1 << 28)):
        assert r(**bad) == SHAPE, bad
    for dims in ((66,), (32, 34), (16, 16, 16, 18), (7,), (0,), (-2, 4), (3, 3)):
        assert r(rotation=turn(dims)) == SHAPE, dims
    assert r(rotation=turn(n=-1)) == SHAPE
    assert r(norm=2) == r(norm=3) == r(norm=-1) == r(rotation=turn(layout=2)) == r(rotation=turn(layout=-1)) == VARIANT
    assert r(t=0) == r(t=0, x=None, out=None, rotation=turn(positions=None)) == OK
    assert r(x=None) == r(out=None) == r(rotation=turn(positions=None)) == r(rotation=turn(freqs=None)) == NULL
    assert r(x=A + 8) == r(out=C + 2) == r(w=B + 2) == ALIGN
    assert r(rotation=turn(positions=I + 2)) == r(rotation=turn(freqs=J + 4)) == ALIGN
    assert r(out=A + 512) == r(out=A, os_=264) == r(out=B - 16) == ALIAS
    assert r(out=A + 256, os_=512, xs=512) == ALIAS      # columns that touch
    assert r(out=I, rotation=turn()) == r(out=J, rotation=turn()) == ALIAS


def test_rope_sizes_reach_the_launch(lib):
    """What is allowed gets as far as the launch, which has no device here."""
    if torch.cuda.is_available():
        pytest.skip("addresses are not real")
    for ok in (dict(), dict(rotation=turn()), dict(rotation=turn((64,), layout=1)), dict(out=A), dict(w=None),
               dict(out=A + 512, xs=512, os_=512), dict(norm=0, w=A + 8), dict(dim=8, heads=1, xs=8, os_=8),
               dict(rotation=turn((2,))), dict(rotation=turn(n=0, layout=9, positions=None))):
        assert rope(lib, **ok) == HIP, ok


def append(lib, q=A, qs=512, hq=4, qw=None, qo=B, qos=256, k=C, ks=512, v=D, vs=512, t=4, hk=2, dim=64, norm=1, kw=None,
           eps=1e-6, rotation=None, at=E, n=64, kc=F, ksc=G, vc=H, vsc=H + (1 << 20)):
    return lib.kq_cache_write_rope(q, qs, hq, qw, qo, qos, k, ks, v, vs, t, hk, dim, norm, kw, eps, rotation, at, n, kc, ksc,
                                   vc, vsc, None)


def test_append_checks(lib):
    a = lambda **kw: append(lib, **kw)
    for bad in (dict(t=-1), dict(hk=0), dict(hk=1, dim=40), dict(hq=0), dict(hq=-3), dict(dim=130), dict(n=-1), dict(n=1 << 31),
                dict(ks=120), dict(vs=68), dict(qs=252), dict(qos=248), dict(eps=-0.5), dict(hk=3, dim=24),
                dict(rotation=turn((68,)))):
        assert a(**bad) == SHAPE, bad
    assert a(norm=2) == a(norm=7) == a(rotation=turn(layout=5)) == VARIANT
    assert a(t=0) == a(t=0, k=None, q=None) == OK
    assert a(n=0, q=None) == OK  # every token is without a slot and nothing else is asked for
    for p in ("qo", "k", "at", "kc", "ksc", "vc", "vsc"):
        assert a(**{p: None}) == NULL, p
    for p, by in (("q", 8), ("qo", 4), ("k", 2), ("v", 8), ("at", 2), ("kc", 8), ("ksc", 2), ("vc", 4), ("vsc", 1)):
        base = dict(q=A, qo=B, k=C, v=D, at=E, kc=F, ksc=G, vc=H, vsc=H + (1 << 20))[p]
        assert a(**{p: base + by}) == ALIGN, p
    assert a(qw=I + 1) == a(kw=I + 2) == ALIGN
    assert a(kc=C) == a(vsc=E) == a(vc=F) == a(ksc=A) == a(qo=F) == a(qo=E) == a(kc=B) == a(kw=F) == a(qw=B) == ALIAS
    assert a(qo=C) == a(qo=D) == ALIAS                       # queries onto keys or values
    assert a(qo=A, qos=520) == ALIAS                         # in place at another stride
    assert a(rotation=turn(positions=F)) == a(rotation=turn(freqs=B)) == ALIAS
    # columns of one matrix: queries, keys and values of a fused projection, the queries turned in place
    fused = dict(q=A, k=A + 512, v=A + 768, qs=512, ks=512, vs=512)
    assert a(**fused, qo=A + 16, qos=512) == a(**fused, qo=A + 128, qos=512) == ALIAS
    if not torch.cuda.is_available():
        assert a(**fused, qo=A, qos=512) == a(**fused) == a(q=None, qo=None, hq=0) == a(v=None, vc=None, vsc=None) == HIP
        assert a(q=None, hq=-5, qs=3) == a(rotation=turn((32, 32), layout=1)) == HIP


def resnorm(lib, x=A, xs=96, y=B, ys=96, t=4, d=96, post=1, pw=None, gate=None, a=1.0, out=C, os_=96, pre=1, w=None, ms=None,
            sh=None, per=1, eps=1e-6, h=D, hs=96, c=None, s=None, stats=None):
    return lib.kq_residual_norm(x, xs, y, ys, t, d, post, pw, gate, a, out, os_, pre, w, ms, sh, per, eps, h, hs, c, s, stats,
                                None)


def test_residual_norm_checks(lib):
    r = lambda **kw: resnorm(lib, **kw)
    for bad in (dict(t=-1), dict(t=1 << 28), dict(d=0), dict(d=72), dict(xs=88), dict(ys=100), dict(os_=64), dict(hs=95),
                dict(eps=-1.0), dict(eps=NAN), dict(a=INF), dict(a=NAN), dict(gate=E, per=0), dict(ms=E, per=-2),
                dict(sh=E, per=0), dict(d=(1 << 24) + 32)):
        assert r(**bad) == SHAPE, bad
    assert r(post=3) == r(pre=-1) == r(pre=4) == r(pre=0, stats=E) == VARIANT
    alone = dict(y=None, out=None, post=0)
    assert r(y=None) == r(y=None, out=None) == r(**alone, pw=E) == r(**alone, gate=E) == r(**alone, a=0.5) == VARIANT
    assert r(y=None, post=0) == VARIANT                      # a stream that is not changed has no other place
    assert r(t=0) == r(t=0, x=None) == OK
    assert r(x=None) == r(out=None) == r(c=E) == r(s=E) == r(**alone, h=None) == NULL
    for p in ("x", "y", "out", "h"):
        assert r(**{p: dict(x=A, y=B, out=C, h=D)[p] + 8}) == ALIGN, p
    for p in ("pw", "gate", "w", "ms", "sh"):
        assert r(**{p: E + 4}) == ALIGN, p
    assert r(c=E + 4, s=F) == r(stats=E + 4) == ALIGN
    assert r(x=A, y=A + 192, out=A + 384, h=A + 560, xs=392, ys=392, os_=392, hs=392) == ALIAS
    assert r(out=B) == r(h=A) == r(h=B) == r(h=C) == r(out=A + 16) == r(out=A, os_=104) == ALIAS
    assert r(c=A, s=E) == r(c=E, s=C) == r(c=E, s=E) == r(stats=D) == r(stats=A) == r(pw=C) == r(gate=D) == r(ms=C) == ALIAS
    assert r(c=E, s=F, stats=E) == r(sh=E, c=E, s=F) == r(w=E, stats=E) == ALIAS
    if not torch.cuda.is_available():
        for ok in (dict(), dict(out=A), dict(h=None), dict(c=E, s=F), dict(alone, h=None, stats=E), dict(post=0, pre=0),
                   dict(gate=E, ms=F, sh=G, pw=H, w=I, per=3), dict(per=0), dict(x=A, y=A + 192, xs=192, ys=192),
                   dict(x=A, y=A + 192, out=A + 384, h=A + 592, xs=392, ys=392, os_=392, hs=392),
                   dict(gate=E, per=1 << 40)):
            assert r(**ok) == HIP, ok


def test_binding_refuses_what_does_not_fit():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    at = torch.zeros(4, dtype=torch.int32)
    pools = kq.alloc_cache(9, 64, "cpu")
    with pytest.raises(ValueError):  # not on the GPU
        kq.kq_rope(x, x, 2)
    with pytest.raises(ValueError):
        kq.kq_cache_write_rope(x, x, at, *pools, 2)
    with pytest.raises(ValueError):
        kq.kq_residual_norm(x, x, x)
    with pytest.raises(ValueError):  # 64 columns are not 3 heads
        kq.kq_rope(x, x, 3)
    with pytest.raises(ValueError):
        kq.kq_rope(x, x, 0)


@pytest.mark.parametrize("dims", [(2, 2, 2, 2, 2), (7,), (0, 4), (-2,), (130,)])
def test_rotation_of_impossible_axes(dims):
    with pytest.raises(ValueError):
        kq._rotation(kq.Rotation(None, None, dims), 4, 0)


def test_rope_freqs():
    f = kq.rope_freqs((4, 6), 100.0, "cpu")
    want = torch.tensor([1.0, 100.0 ** -0.5, 1.0, 100.0 ** (-1 / 3), 100.0 ** (-2 / 3)], dtype=torch.float64)
    assert f.dtype == torch.float64 and torch.allclose(f, want, rtol=1e-15, atol=0)


def test_absurd_head_dims(lib):
    """Refused before a product with the number of heads is formed, which would pass 63 bits."""
    for dim in ((1 << 62) + 8, 1 << 62, -(1 << 62), (1 << 60) + 64, (1 << 63) - 8):
        assert rope(lib, heads=1 << 21, dim=dim) == SHAPE
        assert append(lib, hk=1 << 21, dim=dim) == append(lib, hq=1 << 21, dim=dim) == SHAPE
