"""The cache, attention and epilogue operators together, as a transformer block of this library uses them, on an MI355X:
projections by the W4A4 product with bias, keys and values written to a 4-bit cache, attention over it, the output and
MLP products gated into the residual stream.  Each stage is checked in 64 bits from the stage before; then the block runs
captured, on streams of its own, and from several threads."""
import threading

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


class Block:
    """Cross attention to text states of ragged length, then an MLP, over one residual stream."""

    def __init__(self, seed, batch=2, tokens=96, heads=8, dim=72, text=(45, 77), hidden=640):
        g = torch.Generator().manual_seed(seed)
        d = heads * dim
        self.batch, self.tokens, self.heads, self.dim, self.d = batch, tokens, heads, dim, d
        rows = batch * tokens

        def weight(n, k):
            w = (torch.randn((n, k), generator=g) * k ** -0.5).to(torch.bfloat16).to(DEV)
            out = kq.alloc_outputs(w)
            kq.kq_mx_quantize(w, *out)
            return out

        f32 = lambda *s: torch.randn(s, generator=g).to(DEV)
        self.wq, self.wkv, self.wo = weight(d, d), weight(2 * d, d), weight(d, d)
        self.w1, self.w2 = weight(hidden, d), weight(d, hidden)
        self.bq, self.bkv, self.bo, self.b1, self.b2 = f32(d), f32(2 * d), f32(d), f32(hidden), f32(d)
        self.gate1, self.gate2 = f32(batch, d), f32(batch, d)
        self.start = torch.randn((rows, d), generator=g).to(torch.bfloat16).to(DEV)
        longest = max(text)
        self.text = torch.randn((batch * longest, d), generator=g).to(torch.bfloat16).to(DEV)
        self.page = 32
        self.per = -(-longest // self.page)
        n = (batch * self.per + 3) * self.page
        self.table = torch.randperm(batch * self.per + 3, generator=g)[: batch * self.per].reshape(batch, -1).to(torch.int32)
        self.kv_len = torch.tensor(text, dtype=torch.int32)
        self.slots = torch.full((batch, longest), -1, dtype=torch.int32)  # tokens past a text's length: no slot
        for b in range(batch):
            self.slots[b, : text[b]] = ref.slots_of(self.table, b, text[b], self.page, n).to(torch.int32)
        self.cache = kq.alloc_cache(n, d, DEV)
        e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)
        self.x, self.q, self.kv, self.att, self.h = e(rows, d), e(rows, d), e(batch * longest, 2 * d), e(rows, d), e(rows, hidden)
        self.lse = torch.empty((rows, heads), device=DEV)
        self.codes = {k: kq.alloc_outputs(t) for k, t in (("x", self.x), ("text", self.text), ("att", self.att), ("h", self.h))}
        self.xs = {}
        self.dev = {k: getattr(self, k).to(DEV) for k in ("table", "kv_len", "slots")}

    def quant(self, name, t):
        kq.kq_mx_quantize(t, *self.codes[name])
        return self.codes[name]

    def run(self, keep=False):
        d, T = self.d, self.tokens
        self.x.copy_(self.start)
        kq.kq_gemm_mx_ex(*self.quant("text", self.text), *self.wkv, bias=self.bkv, y_bf16=self.kv)
        kq.kq_cache_write(self.kv[:, :d], self.kv[:, d:], self.dev["slots"].view(-1), *self.cache)
        kq.kq_gemm_mx_ex(*self.quant("x", self.x), *self.wq, bias=self.bq, y_bf16=self.q)
        kq.kq_attention_mx(self.q, *self.cache, self.dev["kv_len"], self.att, self.heads, self.heads, page_size=self.page,
                           page_table=self.dev["table"], lse=self.lse)
        kq.kq_gemm_mx_ex(*self.quant("att", self.att), *self.wo, bias=self.bo, gate=self.gate1, rows_per_sample=T,
                         residual=self.x, y_bf16=self.x)
        if keep:
            self.xs["mid"] = self.x.clone()
        kq.kq_gemm_mx_ex(*self.quant("x", self.x), *self.w1, bias=self.b1, act=kq.KQ_ACT_GELU_TANH, y_bf16=self.h)
        kq.kq_gemm_mx_ex(*self.quant("h", self.h), *self.w2, bias=self.b2, gate=self.gate2, rows_per_sample=T,
                         residual=self.x, y_bf16=self.x)

    def outputs(self):
        return [t.clone() for t in (self.x, self.att, self.lse, self.kv, *self.cache)]


def test_each_stage_of_a_block():
    b = Block(1)
    b.run(keep=True)
    torch.cuda.synchronize()

    def product(t, w, bias, act="none", gate=None, residual=None):
        a = ref.quantize(t.cpu())
        cpu = lambda v: None if v is None else v.cpu()
        return ref.gemm(*a, w[0].cpu(), w[1].cpu(), cpu(bias), act, cpu(gate), b.tokens, cpu(residual))

    def close(got, want, tol):  # a value within the fp32 bound, rounded once to bf16
        got = got.cpu().double()
        assert ((got - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()

    close(b.kv, *product(b.text, b.wkv, b.bkv))
    close(b.q, *product(b.start, b.wq, b.bq))
    at = b.slots.view(-1)
    there = at >= 0
    for x, codes, scales in ((b.kv[:, : b.d], *b.cache[:2]), (b.kv[:, b.d:], *b.cache[2:])):
        want = ref.quantize(x.cpu())
        assert torch.equal(codes.cpu()[at[there].long()], want[0][there])
        assert torch.equal(scales.cpu()[at[there].long()], want[1][there])
        rest = torch.ones(codes.shape[0], dtype=torch.bool)
        rest[at[there].long()] = False
        assert not codes.cpu()[rest].any()
    starts = [i * b.tokens for i in range(b.batch + 1)]
    ref.check_attention(b.att, b.lse, ref.attention(b.q.cpu(), [t.cpu() for t in b.cache], b.kv_len, b.table, b.page,
                                                    b.heads, b.heads, starts))
    close(b.xs["mid"], *product(b.att, b.wo, b.bo, gate=b.gate1, residual=b.start))
    close(b.h, *product(b.xs["mid"], b.w1, b.b1, act="gelu_tanh"))
    close(b.x, *product(b.h, b.w2, b.b2, gate=b.gate2, residual=b.xs["mid"]))


def test_prompt_in_chunks_then_tokens():
    """A causal sequence written and attended in chunks, then token by token, sees what one pass over it sees."""
    heads, kv_heads, dim, page, n = 8, 2, 64, 16, 90
    W = kv_heads * dim
    q, k, v = ref.bf16((n, heads * dim), 1).to(DEV), ref.bf16((n, W), 2).to(DEV), ref.bf16((n, W), 3).to(DEV)
    table = torch.randperm(9, generator=torch.Generator().manual_seed(4))[:6].reshape(1, 6).to(torch.int32)
    cache = kq.alloc_cache(9 * page, W, DEV)
    slots = ref.slots_of(table, 0, n, page, 9 * page).to(torch.int32).to(DEV)
    out, lse = torch.empty_like(q), torch.empty((n, heads), device=DEV)
    at = 0
    for m in [50, 33] + [1] * 7:
        kq.kq_cache_write(k[at:at + m], v[at:at + m], slots[at:at + m], *cache)
        lens = torch.tensor([at + m], dtype=torch.int32, device=DEV)
        kq.kq_attention_mx(q[at:at + m], *cache, lens, out[at:at + m], heads, kv_heads, page_size=page,
                           page_table=table.to(DEV), causal=True, lse=lse[at:at + m])
        at += m
    torch.cuda.synchronize()
    lens = torch.tensor([n], dtype=torch.int32)
    ref.check_attention(out, lse, ref.attention(q.cpu(), [t.cpu() for t in cache], lens, table, page, heads, kv_heads,
                                                [0, n], causal=True))


class Tokens:
    """A decode step whose attention divides its keys and so needs a workspace."""

    def __init__(self, seed):
        self.heads, self.kv_heads, dim, self.page, n = 8, 2, 128, 64, 3000
        W = self.kv_heads * dim
        self.q = ref.bf16((2, self.heads * dim), seed).to(DEV)
        self.cache = kq.alloc_cache(2 * 50 * self.page, W, DEV)
        slots = torch.arange(self.cache[0].shape[0], dtype=torch.int32, device=DEV)
        x = ref.bf16((slots.numel(), 2 * W), seed + 1).to(DEV)
        kq.kq_cache_write(x[:, :W], x[:, W:], slots, *self.cache)
        self.lens = torch.tensor([n, 700], dtype=torch.int32, device=DEV)
        self.out, self.lse = torch.empty_like(self.q), torch.empty((2, self.heads), device=DEV)
        assert kq.kq_attention_mx_workspace(2, 2, 1, self.heads, self.kv_heads, dim, 50 * self.page) > 0

    def run(self, **kw):
        kq.kq_attention_mx(self.q, *self.cache, self.lens, self.out, self.heads, self.kv_heads, page_size=self.page,
                           causal=True, lse=self.lse, **kw)

    def outputs(self):
        return [self.out.clone(), self.lse.clone()]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def capture(thing):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        thing.run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        thing.run()
    torch.cuda.synchronize()
    return g


@pytest.mark.parametrize("kind", [Block, Tokens])
def test_captured_and_replayed(kind):
    """Two captured graphs (each with workspaces of its own) replayed in turn, with eager calls of the same kind between."""
    a, b, other = kind(11), kind(12), kind(13)
    want = []
    for t in (a, b, other):
        t.run()
        torch.cuda.synchronize()
        want.append(t.outputs())
    ga, gb = capture(a), capture(b)
    for _ in range(3):
        for t in (a, b):
            for o in (t.x, t.att, t.lse) if kind is Block else (t.out, t.lse):
                o.zero_()
        ga.replay()
        gb.replay()
        other.run()
        torch.cuda.synchronize()
        assert same(a.outputs(), want[0]) and same(b.outputs(), want[1]) and same(other.outputs(), want[2])


def test_a_stream_that_is_not_the_current_one():
    """stream=: the launches and the workspace's memory belong to that stream, whatever the current one does next."""
    things = [Tokens(20 + i) for i in range(4)]
    want = []
    for t in things:
        t.run()
        torch.cuda.synchronize()
        want.append(t.outputs())
        t.out.zero_()
    streams = [torch.cuda.Stream() for _ in things]
    torch.cuda.synchronize()
    for i, (t, s) in enumerate(zip(things, streams)):
        for _ in range(3):
            t.run(stream=s if i % 2 else s.cuda_stream)
            torch.empty(1 << 20, dtype=torch.uint8, device=DEV).fill_(0xFF)  # the current stream's allocations
    torch.cuda.synchronize()
    assert all(same(t.outputs(), w) for t, w in zip(things, want))


def test_the_default_stream_by_address():
    """stream=0 is the default stream, also from inside another one."""
    t = Tokens(25)
    t.run()
    torch.cuda.synchronize()
    want = t.outputs()
    t.out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        t.run(stream=0)
    torch.cuda.synchronize()
    assert same(t.outputs(), want)


def test_threads_on_their_own_streams():
    things = [Tokens(30), Block(31), Tokens(32), Block(33)]
    want = []
    for t in things:
        t.run()
        torch.cuda.synchronize()
        want.append(t.outputs())
    streams, errors = [torch.cuda.Stream() for _ in things], []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(5):
                    things[i].run()
        except Exception as e:  # reported below, in the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(things))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert all(same(t.outputs(), w) for t, w in zip(things, want))


def test_a_workspace_of_ones_own():
    t = Tokens(40)
    t.run()
    torch.cuda.synchronize()
    want = t.outputs()
    need = kq.kq_attention_mx_workspace(2, 2, 1, 8, 2, 128, 50 * 64)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN wherever nothing was written
    t.run(workspace=ws)
    torch.cuda.synchronize()
    assert same(t.outputs(), want) and (ws[need:] == 0xFF).all()
    with pytest.raises(kq.KQError) as e:
        t.run(workspace=ws[: need - 16])
    assert e.value.status == 7
