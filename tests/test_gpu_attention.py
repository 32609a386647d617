"""kq_attention_mx on an MI355X against attention in 64 bits: lengths from none to thousands, every head layout and
width, pages that end inside a tile, masks that leave rows empty, and buffers that hold anything where nothing is named."""
import math

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


class Case:
    """Queries and a cache whose unnamed slots hold bytes of all ones (scale 255 reads as NaN)."""

    def __init__(self, q_len, kv_len, q_heads, kv_heads, dim, page, seed=0, spare=0, bad=(), peak=1.0, tail=0):
        b = len(kv_len)
        self.heads, self.kv_heads, self.dim, self.page = q_heads, kv_heads, dim, page
        self.q_start = [sum(q_len[:i]) for i in range(b + 1)]
        self.rows = self.q_start[-1] + tail
        self.q = ref.bf16((self.rows, q_heads * dim), seed + 1, peak)
        self.kv_len = torch.tensor(kv_len, dtype=torch.int32)
        self.per = max(1, -(-max(kv_len) // page)) + spare
        pages = b * self.per + 2
        g = torch.Generator().manual_seed(seed)
        self.table = torch.randperm(pages, generator=g)[: b * self.per].reshape(b, self.per).to(torch.int32)
        width = kv_heads * dim
        self.cache = [torch.full((pages * page, w), 0xFF, dtype=torch.uint8) for w in (width // 2, width // 32) * 2]
        for i in range(b):
            at = ref.slots_of(self.table, i, kv_len[i], page, pages * page)
            for j, s in ((0, 2), (2, 3)):
                x = ref.bf16((kv_len[i], width), 10 * seed + 100 * i + s)
                if kv_len[i]:
                    self.cache[j][at], self.cache[j + 1][at] = ref.quantize(x)
        for i, p, to in bad:  # pages that the cache does not have
            self.table[i, p] = to

    def reference(self, **kw):
        return ref.attention(self.q, self.cache, self.kv_len, self.table, self.page, self.heads, self.kv_heads,
                             self.q_start, **kw)

    def run(self, ragged=True, lse=True, **kw):
        d = lambda t: t.to(DEV)
        out = torch.full((self.rows, self.heads * self.dim), 7.0, dtype=torch.bfloat16, device=DEV)
        ls = torch.full((self.rows, self.heads), 7.0, device=DEV) if lse else None
        starts = torch.tensor(self.q_start, dtype=torch.int32)
        longest = int((starts[1:] - starts[:-1]).max())
        kq.kq_attention_mx(d(self.q), *map(d, self.cache), d(self.kv_len), out, self.heads, self.kv_heads,
                           page_size=self.page, page_table=d(self.table), q_start=d(starts) if ragged else None,
                           max_q=longest, lse=ls, **kw)
        torch.cuda.synchronize()
        return out, ls

    def check(self, run=None, **kw):
        run = run or {}
        r = self.reference(**kw)
        out, lse = self.run(**kw, **run)
        ref.check_attention(out, lse, r)
        owned = r[4]
        assert (out[~owned.to(DEV)] == 7).all() and (lse[~owned.to(DEV)] == 7).all()  # rows of no sequence


@pytest.mark.parametrize("dim", [8, 16, 24, 32, 40, 64, 72, 80, 96, 112, 128])
@pytest.mark.parametrize("q_len,kv", [(1, 77), (150, 139)])
def test_head_widths(dim, q_len, kv):
    kv_heads = {8: 4, 16: 2, 24: 4, 40: 4, 72: 4, 80: 2, 112: 2}.get(dim, 1)
    Case([q_len], [kv], 2 * kv_heads, kv_heads, dim, 16, seed=dim).check()


@pytest.mark.parametrize("dim", [8, 32, 40, 64, 72, 96, 104, 128])
def test_few_rows_over_some_hundreds_of_keys(dim):
    """Key sets that are not divided, with every wave of a workgroup at work and with some idle; an empty one."""
    Case([2, 2, 1, 2], [900, 260, 0, 129], 8, 4, dim, 48, seed=dim + 1, bad=[(0, 7, 10 ** 6)]).check(causal=True)


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (3, 1), (8, 2), (32, 1), (5, 5), (48, 3)])
@pytest.mark.parametrize("q_len", [1, 2, 37])
def test_head_groups(q_heads, kv_heads, q_len):
    Case([q_len, 1], [65, 300], q_heads, kv_heads, 64, 64, seed=q_heads).check(causal=True)


@pytest.mark.parametrize("kv", [0, 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 1000, 4097])
@pytest.mark.parametrize("q_len", [1, 33])
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(kv, q_len, causal):
    Case([q_len], [kv], 2, 1, 64, 48, seed=kv).check(causal=causal)


@pytest.mark.parametrize("causal", [False, True])
def test_more_tiles_than_the_gpu_holds(causal):
    """Row tiles that run whole and, of the last, partial round, some whose keys are divided; sequences by length."""
    Case([40] * 13, [130, 300, 0, 64, 257, 300, 1, 129, 290, 31, 200, 299, 128], 20, 20, 8, 16, seed=41).check(causal=causal)
    Case([300, 7, 120], [70, 333, 128], 100, 100, 8, 16, seed=42).check(causal=causal)
    Case([40] * 7, [600, 300, 0, 64, 257, 513, 129], 40, 40, 8, 16, seed=43).check(causal=causal)


@pytest.mark.parametrize("page", [1, 3, 16, 50, 64, 300])
def test_pages_that_end_inside_a_tile(page):
    Case([5, 130], [333, 290], 4, 2, 64, page, seed=page).check(causal=True)
    Case([1, 1], [333, 290], 4, 2, 64, page, seed=page).check(causal=True)


@pytest.mark.parametrize("q_len", [[1, 1, 1, 1, 1], [1, 40, 3, 0, 200]])
@pytest.mark.parametrize("causal", [False, True])
def test_ragged_batches_and_empty_sequences(q_len, causal):
    """Sequences without keys, without queries, and (causal) with fewer keys than queries; rows behind the last."""
    Case(q_len, [700, 64, 0, 31, 5], 8, 2, 128, 16, seed=3, tail=3).check(causal=causal)


@pytest.mark.parametrize("dim,kv", [(32, 512), (64, 512), (64, 513), (72, 320), (72, 321), (112, 256), (128, 256), (128, 257)])
@pytest.mark.parametrize("causal", [False, True])
def test_around_what_local_memory_holds(dim, kv, causal):
    """Keys that just fit beside one another on chip, and one more; several groups of rows to a workgroup."""
    kv_heads = 4 if dim in (72, 112) else 1
    Case([600, 33], [kv, kv - 65], kv_heads, kv_heads, dim, 16, seed=dim, tail=1).check(causal=causal)


def test_many_rows_over_few_keys():
    """Enough rows that a workgroup takes several runs of them: 8 x 1111 rows of 24 heads over up to 70 keys."""
    c = Case([1111] * 8, [70, 1, 0, 64, 65, 33, 17, 69], 24, 24, 64, 70, seed=51)
    c.check()


def test_uniform_batch_without_table_or_starts():
    c = Case([6, 6, 6], [40, 1, 64], 4, 4, 72, 64, seed=5)
    c.table = torch.arange(3, dtype=torch.int32)[:, None]
    n = 3 * 64
    for j, (x, s) in enumerate(((0, 21), (2, 22))):
        c.cache[x], c.cache[x + 1] = ref.quantize(ref.bf16((n, 4 * 72), s))
    r = c.reference()
    out = torch.empty((18, 4 * 72), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((18, 4), device=DEV)
    kq.kq_attention_mx(c.q.to(DEV), *[t.to(DEV) for t in c.cache], c.kv_len.to(DEV), out, 4, 4, lse=lse)
    ref.check_attention(out, lse, r)


@pytest.mark.parametrize("dim,spare", [(40, 0), (64, 0), (128, 0), (64, 400), (72, 400), (128, 400)])
@pytest.mark.parametrize("q_len", [1, 3])
def test_few_rows_over_divided_keys(dim, spare, q_len):
    """A ragged batch whose key ranges are joined; with spare pages, room enough that a workgroup takes two heads."""
    Case([q_len] * 6, [4600, 0, 2049, 1, 300, 3000], 8, 4, dim, 64 if spare == 0 else 128, seed=dim, spare=spare,
         bad=[(0, 20, -1)]).check(causal=True)


@pytest.mark.parametrize("q_len", [1, 140])
def test_pages_outside_the_cache_are_masked(q_len):
    c = Case([q_len] * 3, [200, 64, 33], 4, 2, 64, 32, seed=7,
             bad=[(0, 1, -1), (0, 3, 10 ** 6), (1, 0, -2 ** 31), (1, 1, 2 ** 31 - 1), (2, 1, -5)])
    c.check()
    c.check(causal=True)


@pytest.mark.parametrize("q_len,kv", [(1, 2000), (4, 500), (130, 700)])
def test_sharp_and_flat_distributions(q_len, kv):
    """Scores of some hundreds (one key takes all), and a scale so small that every key counts alike."""
    Case([q_len], [kv], 4, 2, 128, 64, seed=11, peak=60.0).check()
    Case([q_len], [kv], 4, 2, 128, 64, seed=12).check(scale=2.0 ** -20)


def test_repeated_pages_and_long_tables():
    c = Case([3, 3], [256, 256], 4, 1, 64, 64, seed=13, spare=60)
    c.table[1, :4] = c.table[0, :4]  # a shared prompt
    c.check(causal=True)


@pytest.mark.parametrize("q_len", [1, 70])
def test_strided_queries_and_outputs(q_len):
    """Queries and outputs as columns of wider matrices."""
    c = Case([q_len, q_len], [90, 10], 4, 2, 64, 16, seed=17)
    r = c.reference()
    wide = torch.randn((c.rows, 3 * 256), device=DEV).to(torch.bfloat16)
    wide[:, 256:512] = c.q.to(DEV)
    out = torch.full((c.rows, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((c.rows, 4), device=DEV)
    kq.kq_attention_mx(wide[:, 256:512], *[t.to(DEV) for t in c.cache], c.kv_len.to(DEV), out[:, :256], 4, 2,
                       page_size=16, page_table=c.table.to(DEV), lse=lse)
    ref.check_attention(out[:, :256], lse, r)
    assert (out[:, 256:] == 7).all()


def test_lengths_and_starts_are_cut():
    """Lengths past the table or below zero and ranges past the queries, as the header says they are read."""
    c = Case([4, 4], [64, 64], 2, 1, 64, 64, seed=19)
    d = [t.to(DEV) for t in c.cache]
    lens = torch.tensor([10 ** 9, -3], dtype=torch.int32)
    starts = torch.tensor([0, 4, 10 ** 9], dtype=torch.int32)
    out = torch.empty((8, 128), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((8, 2), device=DEV)
    kq.kq_attention_mx(c.q.to(DEV), *d, lens.to(DEV), out, 2, 1, page_size=64, page_table=c.table.to(DEV),
                       q_start=starts.to(DEV), max_q=8, lse=lse)
    c.kv_len = torch.tensor([64, 0], dtype=torch.int32)
    ref.check_attention(out, lse, c.reference())


def test_queries_past_max_q_are_left():
    c = Case([6, 6], [64, 64], 2, 1, 64, 64, seed=23)
    out = torch.full((12, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((12, 2), 7.0, device=DEV)
    kq.kq_attention_mx(c.q.to(DEV), *[t.to(DEV) for t in c.cache], c.kv_len.to(DEV), out, 2, 1, page_size=64,
                       page_table=c.table.to(DEV), q_start=torch.tensor(c.q_start, dtype=torch.int32, device=DEV),
                       max_q=4, causal=True, lse=lse)
    r = [t.clone() for t in c.reference(causal=True)]
    left = torch.tensor([4, 5, 10, 11])
    r[4][left] = False
    ref.check_attention(out, lse, r)
    assert (out[left.to(DEV)] == 7).all() and (lse[left.to(DEV)] == 7).all()


def test_a_query_that_is_not_finite_stays_alone():
    for q_len in (8, 140):
        c = Case([q_len], [100], 2, 1, 64, 64, seed=29)
        r = c.reference()
        c.q[3] = math.nan
        out, lse = c.run()
        keep = torch.ones(q_len, dtype=torch.bool)
        keep[3] = False
        r[4][3] = False
        assert torch.isnan(out[3]).all()
        lse[3] = 0.0
        r[1][3] = 0.0
        r[3][3] = 1.0
        ref.check_attention(out, lse, r)


def test_same_bits_each_time_and_without_lse():
    for q_len, kv in (([1, 1], [3000, 17]), ([200, 70], [400, 400])):
        c = Case(q_len, kv, 8, 2, 128, 64, seed=31)
        a, _ = c.run(causal=True)
        b, _ = c.run(causal=True, lse=False)
        assert torch.equal(a, b)


def test_cache_past_4_gib():
    """Keys at slots whose codes start beyond byte 2^32."""
    width, n, page = 4096, 2_200_000, 100
    cache = tuple(torch.empty((n, w), dtype=torch.uint8, device=DEV) for w in (2048, 128, 2048, 128))
    table = torch.tensor([[21_000, 3, 21_999]], dtype=torch.int32)
    at = ref.slots_of(table, 0, 250, page, n).to(DEV)
    k, v = ref.bf16((250, width), 1), ref.bf16((250, width), 2)
    kq.kq_cache_write(k.to(DEV), v.to(DEV), at.to(torch.int32), *cache)
    for q_len in (1, 40):
        q = ref.bf16((q_len, width), 3)
        out = torch.empty((q_len, width), dtype=torch.bfloat16, device=DEV)
        lse = torch.empty((q_len, 32), device=DEV)
        lens = torch.tensor([250], dtype=torch.int32)
        kq.kq_attention_mx(q.to(DEV), *cache, lens.to(DEV), out, 32, 32, page_size=page, page_table=table.to(DEV), lse=lse)
        small = [t[at].cpu() for t in cache]  # the same keys in order
        ref.check_attention(out, lse, ref.attention(q, small, lens, torch.zeros((1, 1), dtype=torch.int32), 250, 32, 32,
                                                    [0, q_len]))


@pytest.mark.parametrize("q_len", [1, 40])
def test_a_cache_without_room(q_len):
    """No pages to a sequence, or none in the cache that is whole: every query is empty."""
    q = ref.bf16((2 * q_len, 128), 1).to(DEV)
    lens = torch.tensor([5, 10 ** 6], dtype=torch.int32, device=DEV)
    for per, n_slots in ((0, 64), (3, 15)):
        cache = [torch.full((n_slots, w), 0xFF, dtype=torch.uint8, device=DEV) for w in (32, 2, 32, 2)]
        table = torch.zeros((2, per), dtype=torch.int32, device=DEV)
        out = torch.full((2 * q_len, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.zeros((2 * q_len, 2), device=DEV)
        kq.kq_attention_mx(q, *cache, lens, out, 2, 1, page_size=16, page_table=table, lse=lse)
        assert not out.any() and torch.isneginf(lse).all()
