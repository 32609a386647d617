"""kq_attention_mx on an MI355X where its ways of dividing the work meet values, batches and calls at their limits."""
import pytest
import torch

import cache_reference as ref
from test_gpu_attention import DEV, Case

kq = pytest.importorskip("w4a4_diffusion_transformer_amd")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    kq.lib()


def workspace(c, q_len):
    return kq.kq_attention_mx_workspace(c.rows, len(c.kv_len), max(q_len), c.heads, c.kv_heads, c.dim, c.per * c.page)


# queries, keys, heads, key heads, channels, spare pages, whether key ranges are joined
NAN_CASES = [([1, 1], [3000, 17], 8, 2, 128, 0, True),         # few rows, a head a workgroup
             ([1, 1, 1], [4600, 2049, 300], 8, 4, 64, 4000, True),  # two heads a workgroup
             ([2, 1], [3000, 900], 8, 4, 72, 4000, True),
             ([3, 2], [100, 64], 4, 2, 64, 0, False),          # whole, four waves
             ([2, 2], [900, 260], 8, 4, 40, 0, False),         # whole, eight
             ([140, 30], [700, 600], 4, 2, 64, 0, True),       # many rows
             ([140, 30], [100, 70], 4, 2, 64, 0, False)]       # many rows, keys on chip


@pytest.mark.parametrize("q_len,kv,q_heads,kv_heads,dim,spare,joined", NAN_CASES)
@pytest.mark.parametrize("causal", [False, True])
def test_a_nan_query_gives_nan_and_stays_alone(q_len, kv, q_heads, kv_heads, dim, spare, joined, causal):
    """out and lse of the query are NaN, however its keys are divided, and no other query's change."""
    c = Case(q_len, kv, q_heads, kv_heads, dim, 64 if spare == 0 else 128, seed=61, spare=spare)
    assert (workspace(c, q_len) > 0) == joined
    r = [t.clone() for t in c.reference(causal=causal)]
    row = q_len[0] - 1  # the first sequence's last query
    c.q[row] = float("nan")
    out, lse = c.run(causal=causal)
    assert torch.isnan(out[row]).all() and torch.isnan(lse[row]).all()
    lse[row], r[1][row] = 0.0, 0.0
    r[4][row] = False
    ref.check_attention(out, lse, r)


@pytest.mark.parametrize("q_len,q_heads,kv_heads,dim,first,last,kv", [
    ([1], 8, 2, 64, 64, 128, 130),      # all that one wave of a whole key set has
    ([1], 8, 2, 128, 0, 3000, 3000),    # every key of a divided one
    ([1], 8, 2, 128, 2990, 3000, 3000),
    ([140], 4, 2, 64, 64, 128, 700), ([140], 4, 2, 64, 0, 64, 100)])
def test_nan_keys_reach_every_query_that_sees_them(q_len, q_heads, kv_heads, dim, first, last, kv):
    c = Case(q_len, [kv], q_heads, kv_heads, dim, 64, seed=62)
    at = ref.slots_of(c.table, 0, kv, 64, c.cache[0].shape[0])[first:last]
    c.cache[1][at] = 0xFF  # key scales that read as NaN
    out, lse = c.run()
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("form", ["object", "address", "default object", "default address"])
def test_the_workspace_belongs_to_the_stream_that_uses_it(form, monkeypatch):
    """Memory that torch keeps for that stream: freed on return, it is next used by work behind the call."""
    c = Case([1, 1], [3000, 17], 8, 2, 128, 64, seed=63)
    assert workspace(c, [1]) > 0
    r = c.reference()
    s = torch.cuda.default_stream() if "default" in form else torch.cuda.Stream()
    owners, empty = [], torch.empty

    def recorded(*args, **kw):
        owners.append(torch.cuda.current_stream().cuda_stream)
        return empty(*args, **kw)

    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda.synchronize()
        monkeypatch.setattr(torch, "empty", recorded)
        inputs = [t.to(DEV) for t in (c.q, *c.cache, c.kv_len, c.table)]
        out, lse = empty((2, 8 * 128), dtype=torch.bfloat16, device=DEV), empty((2, 8), device=DEV)
        torch.cuda.synchronize()
        owners.clear()
        kq.kq_attention_mx(*inputs[:6], out, 8, 2, page_size=64, page_table=inputs[6], lse=lse,
                           stream=s.cuda_stream if "address" in form else s)
        monkeypatch.undo()
        torch.cuda.synchronize()
    assert owners == [s.cuda_stream] and (s.cuda_stream == 0) == ("default" in form)
    ref.check_attention(out, lse, r)


@pytest.mark.parametrize("causal", [False, True])
def test_more_sequences_than_are_ranked(causal):
    """65 sequences and more start in their own order, of many rows, the last round divided, and of few."""
    for n, heads, kv_heads, q, most in ((67, 4, 4, 40, 600), (96, 8, 4, 20, 530), (200, 8, 2, 1, 2300),
                                        (130, 4, 1, 2, 4100)):
        kv = [(37 * i * i + 11) % most for i in range(n - 1)] + [most]
        q_len = [q - (i % 3 if q > 2 else 0) for i in range(n)]
        c = Case(q_len, kv, heads, kv_heads, 8 if q > 2 else 32, 16, seed=n)
        assert workspace(c, q_len) > 0, n
        c.check(causal=causal)


@pytest.mark.parametrize("q_len", [1, 40])
def test_the_default_share_of_a_cache(q_len):
    """Without a table or a page size each sequence has an equal share: of more slots than a page may have (2^24), and
    of fewer slots than there are sequences, where every query is empty."""
    for n, batch in (((1 << 24) + 70, 1), (2 * (1 << 24) + 131, 2), (2, 3)):
        cache = [torch.zeros((n, w), dtype=torch.uint8, device=DEV) for w in (16, 1, 16, 1)]
        share = n // batch
        kv_len = torch.tensor([min(share, 333 + i) for i in range(batch)], dtype=torch.int32)
        for i in range(batch if share else 0):
            at = torch.arange(kv_len[i]) + i * share
            for j, s in ((0, 1), (2, 2)):
                codes, scales = ref.quantize(ref.bf16((len(at), 32), 10 * i + s))
                cache[j][at.to(DEV)], cache[j + 1][at.to(DEV)] = codes.to(DEV), scales.to(DEV)
        q = ref.bf16((batch * q_len, 64), 3)
        out = torch.full((batch * q_len, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((batch * q_len, 2), 7.0, device=DEV)
        kq.kq_attention_mx(q.to(DEV), *cache, kv_len.to(DEV), out, 2, 1, lse=lse)
        if share == 0:
            assert not out.any() and torch.isneginf(lse).all()
            continue
        small = torch.cat([torch.arange(333 + batch) + i * share for i in range(batch)]).to(DEV)  # the slots that have keys
        table = torch.arange(batch, dtype=torch.int32)[:, None]
        ref.check_attention(out, lse, ref.attention(q, [t[small].cpu() for t in cache], kv_len, table, 333 + batch, 2, 1,
                                                    [i * q_len for i in range(batch + 1)]))
