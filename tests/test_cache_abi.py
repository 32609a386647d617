"""Refusals of the cache, attention and epilogue entry points, without a GPU: the C ABI returns before any HIP call,
the binding raises on tensors that do not fit one another."""
import ctypes
import os

import pytest
import torch

import w4a4_diffusion_transformer_amd as kq

OK, NULL, SHAPE, ALIGN, VARIANT, HIP, ALIAS, WORKSPACE = range(8)
A, B, C, D, E, F, G, H = (i << 28 for i in range(1, 9))  # aligned fake device addresses


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kq.LIB_PATH):
        pytest.skip("libkq.so not built")
    return kq.lib()


def test_cache_write_checks(lib):
    w = lambda k=A, ks=64, v=B, vs=64, t=4, d=64, at=C, n=16, kc=D, ksc=E, vc=F, vsc=G: lib.kq_cache_write(
        k, ks, v, vs, t, d, at, n, kc, ksc, vc, vsc, None)
    assert w(d=48) == w(d=0) == w(t=-1) == w(t=1 << 28) == w(n=-1) == w(n=1 << 31) == SHAPE
    assert w(ks=56) == w(ks=68) == w(vs=32) == w(ks=1 << 32) == SHAPE
    assert w(t=0) == w(t=0, k=None, at=None, kc=None) == OK
    assert w(n=0) == OK  # every token is without a slot
    assert w(k=None) == w(at=None) == w(kc=None) == w(ksc=None) == w(vc=None) == w(vsc=None) == NULL
    assert w(k=A + 8) == w(kc=D + 8) == w(ksc=E + 2) == w(at=C + 2) == w(v=B + 2) == w(vc=F + 4) == w(vsc=G + 1) == ALIGN
    assert w(kc=A) == w(vsc=C) == w(vc=D) == w(ksc=D + 64) == w(vc=B + 16) == ALIAS


def test_cache_read_checks(lib):
    r = lambda k=A, ks=64, v=B, vs=64, t=4, d=64, at=C, n=16, kc=D, ksc=E, vc=F, vsc=G: lib.kq_cache_read(
        kc, ksc, vc, vsc, n, d, at, t, k, ks, v, vs, None)
    assert r(d=40) == r(t=-1) == r(n=1 << 31) == r(ks=60) == r(vs=63) == SHAPE
    assert r(t=0, k=None) == OK
    assert r(k=None) == r(vsc=None) == NULL
    assert r(v=B + 4) == r(kc=D + 1) == ALIGN
    assert r(k=D) == r(v=E) == r(v=C - 16) == ALIAS
    assert r(v=A + 64) == r(v=A) == ALIAS                    # rows of 64 that touch
    assert r(ks=128, vs=128, v=A + 64) == ALIAS              # columns 32 .. of a matrix whose columns 0 .. 63 are K's
    assert r(ks=128, vs=136, v=A + 128) == ALIAS


def test_cache_read_into_columns_in_either_order(lib):
    """K and V as column ranges of one matrix, V above or below K, at strides that are and are not powers of two."""
    r = lambda k, v, w, s: lib.kq_cache_read(D, E, F, G, 16, w, C, 4, k, s, v, s, None)
    for w, s in ((1152, 2304), (64, 136), (64, 128), (1024, 4096), (96, 200)):
        base = A + 16 * s
        # elements from one to the other, no row of them touching; the call gets as far as the launch, so only where
        # that has no device to go to
        for d in () if torch.cuda.is_available() else (w, s - w, 2 * s + w, -s + w):
            assert r(base, base + 2 * d, w, s) == r(base + 2 * d, base, w, s) == HIP, (w, s, d)
        for d in (0, 8, w - 8, s - w + 8, s, s + w - 8, 2 * s - 8):
            assert r(base, base + 2 * d, w, s) == r(base + 2 * d, base, w, s) == ALIAS, (w, s, d)


def attention(lib, q=A, qs=256, rows=8, start=None, batch=2, max_q=4, kc=B, ks=C, vc=D, vs=E, n=256, table=F, per=2,
              page=64, lens=G, hq=4, hk=2, dim=64, scale=0.125, causal=0, out=H, os_=256, lse=None, ws=None, wb=0):
    return lib.kq_attention_mx(q, qs, rows, start, batch, max_q, kc, ks, vc, vs, n, table, per, page, lens, hq, hk, dim,
                               scale, causal, out, os_, lse, ws, wb, None)


def test_attention_checks(lib):
    a = lambda **kw: attention(lib, **kw)
    for bad in (dict(rows=-1), dict(batch=-1), dict(batch=65536), dict(max_q=-1), dict(max_q=9), dict(max_q=5),
                dict(hq=3), dict(hq=0), dict(hk=0), dict(dim=60), dict(dim=136), dict(dim=0), dict(hk=1, dim=40),
                dict(page=0), dict(page=(1 << 24) + 1), dict(per=-1), dict(n=-1), dict(n=1 << 31),
                dict(table=None, n=255), dict(qs=248), dict(qs=260), dict(os_=128), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(per=1 << 20, page=1 << 20)):
        assert a(**bad) == SHAPE, bad
    assert a(batch=0) == a(max_q=0) == a(rows=0, max_q=0) == OK
    for p in ("q", "kc", "ks", "vc", "vs", "lens", "out"):
        assert a(**{p: None}) == NULL, p
    for p, by in (("q", 8), ("out", 2), ("kc", 4), ("vc", 8), ("ks", 2), ("vs", 1), ("lens", 2), ("table", 1),
                  ("start", 2), ("lse", 2), ("ws", 4)):
        base = dict(q=A, out=H, kc=B, vc=D, ks=C, vs=E, lens=G, table=F, start=1 << 20, lse=1 << 20, ws=1 << 20)[p]
        assert a(**{p: base + by}) == ALIGN, p
    big = dict(per=1024, n=1 << 17)
    need = lib.kq_attention_mx_workspace(8, 2, 4, 4, 2, 64, 1 << 16)
    assert need > 0 and lib.kq_attention_mx_workspace(8, 2, 4, 4, 2, 64, 64) == 0
    assert lib.kq_attention_mx_workspace(8, 2, 4, 4, 3, 64, 1 << 16) == 0  # sizes that are refused
    assert a(**big) == a(**big, ws=1 << 20, wb=need - 1) == a(**big, wb=need) == WORKSPACE
    assert a(out=A) == a(out=B) == a(lse=H) == a(lse=G) == a(out=F) == ALIAS
    assert a(**big, ws=A, wb=need) == ALIAS


def test_attention_of_no_sequences(lib):
    """No batch is nothing to do and needs no workspace, at every division of the work."""
    for rows, cap in ((1, 64), (1, 1 << 20), (4096, 64), (4096, 256), (4096, 1 << 20)):
        assert lib.kq_attention_mx_workspace(rows, 0, rows, 4, 2, 64, cap) == 0
        assert attention(lib, rows=rows, batch=0, max_q=rows, per=1, page=cap) == OK


def test_gemm_ex_checks(lib):
    g = lambda a=A, m=4, n=8, k=64, bias=None, act=0, gate=None, rps=1, res=None, yf=None, yb=F: lib.kq_gemm_mx_ex(
        a, B, m, C, D, n, k, bias, act, gate, rps, res, yf, yb, None)
    assert g(act=4) == g(act=-1) == VARIANT
    assert g(k=48) == g(m=-1) == g(n=(1 << 22) + 1) == g(gate=E, rps=0) == g(gate=E, rps=-5) == SHAPE
    assert g(m=0) == g(n=0, gate=E) == OK
    assert g(gate=F + 8, rps=(1 << 63) - 1) == ALIAS  # one sample
    assert g(yb=None) == g(a=None) == NULL
    assert g(bias=E + 2) == g(gate=E + 1) == g(res=E + 1) == ALIGN
    assert g(yb=B) == g(bias=F) == g(gate=F + 8) == g(res=F + 2) == g(yf=E, res=E) == g(yf=F) == ALIAS


def test_status_string(lib):
    assert kq.kq_status_str(WORKSPACE) == "workspace missing or too small"


def test_binding_refuses_what_does_not_fit():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    at = torch.zeros(4, dtype=torch.int32)
    pools = (u8(9, 32), u8(9, 2), u8(9, 32), u8(9, 2))
    with pytest.raises(ValueError):  # not on the GPU
        kq.kq_cache_write(x, x, at, *pools)
    with pytest.raises(ValueError):
        kq.kq_cache_read(*pools, at, x, x)
    with pytest.raises(ValueError):
        kq.kq_gemm_mx_ex(u8(4, 32), u8(4, 2), u8(8, 32), u8(8, 2), y_bf16=x)
    with pytest.raises(ValueError):
        kq.kq_attention_mx(x, *pools, at, x, 2, 2)
    with pytest.raises(ValueError):  # 64 columns are not 3 heads
        kq.kq_attention_mx(x, *pools, at, x, 3, 3)
    with pytest.raises(ValueError):
        kq.kq_attention_mx(x, *pools, at, x, 0, 1)
    with pytest.raises(ValueError):  # a table without its page size
        kq.kq_attention_mx(x, *pools, at, x, 2, 2, page_table=at.reshape(4, 1))


def test_alloc_cache():
    kc, ks, vc, vs = kq.alloc_cache(5, 96, device="cpu")
    assert kc.shape == vc.shape == (5, 48) and ks.shape == vs.shape == (5, 3) and not kc.any()


def test_what_divides_the_keys_of_few_rows(lib):
    """Key ranges of few rows are balanced over the batch by a sum that fits 32 bits for 512 sequences: no more than
    that are ever divided."""
    for batch in (1, 8, 64, 65, 256, 512, 513, 1024, 1025, 65535):
        for kv_heads, group, dim in ((1, 1, 64), (1, 8, 128), (2, 4, 64), (8, 4, 128), (5, 1, 32), (16, 1, 128)):
            for cap in (1, 2047, 1 << 14, 1 << 20, 1 << 30):
                need = lib.kq_attention_mx_workspace(batch, batch, 1, kv_heads * group, kv_heads, dim, cap)
                assert need == 0 or batch <= 512, (batch, kv_heads, cap)
    assert lib.kq_attention_mx_workspace(8, 8, 1, 32, 8, 128, 1 << 14) > 0


def test_attention_past_what_a_launch_holds(lib):
    """Sizes whose launch would have 2^32 threads or more are refused before it; just below, the checks go on."""
    a = lambda b, q, group, heads, per, page: attention(lib, q=A, qs=1 << 20, rows=b * q, batch=b, max_q=q, per=per, page=page,
                                                        n=1 << 20, hq=heads * group, hk=heads, dim=8, os_=1 << 20, lens=None)
    for ok, sizes in ((True, (65535, 1, 1, 508, 1, 64)), (False, (65535, 1, 1, 512, 1, 64)),    # few rows, two heads
                      (True, (65535, 1, 1, 252, 0, 64)), (False, (65535, 1, 1, 256, 0, 64)),   # one head
                      (True, (65535, 1, 36, 60, 1, 64)), (False, (65535, 1, 36, 68, 1, 64)),    # keys on chip
                      (True, (65535, 1, 36, 124, 1, 1024)), (False, (65535, 1, 36, 132, 1, 1024))):
        assert a(*sizes) == (NULL if ok else SHAPE), sizes


def test_attention_scale_and_its_multiple_are_finite(lib):
    """The kernels work in powers of two: scale * log2(e) has to be finite too."""
    for scale in (2.0 ** 127 * 1.001, 2.9e38, 3.2e38, float("inf")):
        assert attention(lib, scale=scale, lens=None) == SHAPE, scale
    for scale in (2.0 ** 127, 1e-30, 1.0):
        assert attention(lib, scale=scale, lens=None) == NULL, scale
