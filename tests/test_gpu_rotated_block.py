"""The rotary, cache-append and residual-norm operators in a transformer block of this library, on an MI355X: the first
block's norm quantised for a fused projection, its queries and keys normalised and turned by the places of a video's
tokens, keys and values to a 4-bit cache, attention over it, and the residual stream carried through sandwich norms.
Each stage is checked in 64 bits from the stage before; then the block runs captured, on streams of its own, from several
threads, and token by token."""
import threading

import pytest
import torch

import block_reference as bref
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
    """Self attention of a guidance batch of videos, then an MLP, over one residual stream, on the plain quantizer."""

    def __init__(self, seed, batch=2, tokens=90, heads=8, kv_heads=4, dim=72, hidden=640, halves=False):
        g = torch.Generator().manual_seed(seed)
        d, W = heads * dim, kv_heads * dim
        self.batch, self.tokens, self.heads, self.kv_heads, self.dim, self.d, self.W = batch, tokens, heads, kv_heads, dim, d, W
        rows = batch * tokens

        def weight(n, k):
            w = (torch.randn((n, k), generator=g) * k ** -0.5).to(torch.bfloat16).to(DEV)
            return kq.kq_mx_quantize(w, *kq.alloc_outputs(w))

        f32 = lambda *s: torch.randn(s, generator=g).to(DEV)
        self.wqkv, self.wo, self.w1, self.w2 = weight(d + 2 * W, d), weight(d, d), weight(hidden, d), weight(d, hidden)
        self.gate1, self.gate2 = f32(batch, d), f32(batch, d)
        self.scale1, self.shift1, self.scale2, self.shift2 = (0.3 * f32(batch, d) for _ in range(4))
        self.norms = [0.5 + f32(d).abs() for _ in range(3)]
        self.wq, self.wk = 0.5 + f32(dim).abs(), 0.5 + f32(dim).abs()
        t = torch.arange(tokens)
        place = torch.stack((t // 30, t // 6 % 5, t % 6), 1).to(torch.int32).repeat(batch, 1)
        axes = (dim - 2 * (dim // 3 // 2 * 2),) + (dim // 3 // 2 * 2,) * 2
        self.turn = (place, kq.rope_freqs(axes, 256.0, "cpu"), axes, halves)
        self.rotation = kq.Rotation(place.to(DEV), self.turn[1].to(DEV), axes, halves)
        self.start = torch.randn((rows, d), generator=g).to(torch.bfloat16).to(DEV)
        self.slots = torch.arange(rows, dtype=torch.int32)
        self.cache = kq.alloc_cache(rows, W, DEV)
        self.kv_len = torch.full((batch,), tokens, dtype=torch.int32)
        e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)
        self.qkv, self.att, self.y1, self.h, self.y2 = e(rows, d + 2 * W), e(rows, d), e(rows, d), e(rows, hidden), e(rows, d)
        self.x, self.q, self.h1 = e(rows, d), e(rows, d), e(rows, d)
        self.lse = torch.empty((rows, heads), device=DEV)
        self.stats = torch.empty((rows, 2), device=DEV)
        self.codes = {k: kq.alloc_outputs(v) for k, v in (("x", self.x), ("att", self.att), ("mid", self.x), ("h", self.h))}
        self.dev = {"slots": self.slots.to(DEV), "kv_len": self.kv_len.to(DEV)}
        self.keep = {}

    def run(self, keep=False):
        d, W, T = self.d, self.W, self.tokens
        self.x.copy_(self.start)
        # the first norm: the stream as it is
        kq.kq_residual_norm(self.x, None, None, pre=kq.KQ_NORM_LAYER, mod_scale=self.scale1, mod_shift=self.shift1,
                            tokens_per_sample=T, h=self.h1, out_codes=self.codes["x"][0], out_scales=self.codes["x"][1])
        kq.kq_gemm_mx_ex(*self.codes["x"], *self.wqkv, y_bf16=self.qkv)
        kq.kq_cache_write_rope(self.qkv[:, d:d + W], self.qkv[:, d + W:], self.dev["slots"], *self.cache, self.kv_heads,
                               rotation=self.rotation, norm=kq.KQ_NORM_RMS, k_weight=self.wk, Q=self.qkv[:, :d], q_out=self.q,
                               q_heads=self.heads, q_weight=self.wq)
        kq.kq_attention_mx(self.q, *self.cache, self.dev["kv_len"], self.att, self.heads, self.kv_heads, lse=self.lse)
        kq.kq_gemm_mx_ex(*kq.kq_mx_quantize(self.att, *self.codes["att"]), *self.wo, y_bf16=self.y1)
        # between attention and MLP: norms on both sides, the stream updated in place
        kq.kq_residual_norm(self.x, self.y1, self.x, post=kq.KQ_NORM_RMS, post_weight=self.norms[0], gate=self.gate1,
                            pre=kq.KQ_NORM_RMS, pre_weight=self.norms[1], mod_scale=self.scale2, mod_shift=self.shift2,
                            tokens_per_sample=T, out_codes=self.codes["mid"][0], out_scales=self.codes["mid"][1])
        if keep:
            self.keep["x1"] = self.x.clone()
        kq.kq_gemm_mx_ex(*self.codes["mid"], *self.w1, act=kq.KQ_ACT_SILU, y_bf16=self.h)
        kq.kq_gemm_mx_ex(*kq.kq_mx_quantize(self.h, *self.codes["h"]), *self.w2, y_bf16=self.y2)
        # after the MLP: the statistics for the next block's quantizer
        kq.kq_residual_norm(self.x, self.y2, self.x, post=kq.KQ_NORM_RMS, post_weight=self.norms[2], gate=self.gate2,
                            tokens_per_sample=T, pre=kq.KQ_NORM_LAYER, row_stats=self.stats)

    def outputs(self):
        return [t.clone() for t in (self.x, self.stats, self.q, self.att, *self.cache, *self.codes["mid"], *self.codes["x"])]


@pytest.mark.parametrize("halves", [False, True])
def test_each_stage_of_a_block(halves):
    b = Block(1, halves=halves)
    b.run(keep=True)
    torch.cuda.synchronize()
    T, d, W = b.tokens, b.d, b.W
    cpu = lambda t: t.cpu()
    h, slack, *_ = bref.following(cpu(b.start), 2, None, cpu(b.scale1), cpu(b.shift1), T)
    bref.check(b.h1, h, slack, what="first norm")
    bref.check_codes(*b.codes["x"], b.h1, "first norm")
    qkv = cpu(b.qkv)
    bref.check(b.q, *bref.rope(qkv[:, :d], b.heads, b.turn, True, cpu(b.wq)), what="queries")
    keys = bref.rounded(bref.rope(qkv[:, d:d + W], b.kv_heads, b.turn, True, cpu(b.wk))[0]).to(torch.bfloat16)
    bref.check_codes(b.cache[0], b.cache[1], keys, "keys")
    bref.check_codes(b.cache[2], b.cache[3], qkv[:, d + W:], "values")
    starts = [i * T for i in range(b.batch + 1)]
    table = torch.arange(b.batch, dtype=torch.int32)[:, None]
    ref.check_attention(b.att, b.lse, ref.attention(cpu(b.q), [cpu(t) for t in b.cache], b.kv_len, table, T, b.heads,
                                                    b.kv_heads, starts))
    x1 = b.keep["x1"]
    bref.check(x1, *bref.residual(cpu(b.start), cpu(b.y1), 1, cpu(b.norms[0]), cpu(b.gate1), per=T), what="stream")
    h, slack, *_ = bref.following(cpu(x1), 1, cpu(b.norms[1]), cpu(b.scale2), cpu(b.shift2), T)
    lo, hi = bref.between(h, slack)
    sure = (lo == hi).all(1)  # rows without a tie
    assert sure.float().mean() > 0.9
    bref.check_codes(cpu(b.codes["mid"][0])[sure], cpu(b.codes["mid"][1])[sure], lo[sure].to(torch.bfloat16), "second norm")
    bref.check(b.x, *bref.residual(cpu(x1), cpu(b.y2), 1, cpu(b.norms[2]), cpu(b.gate2), per=T), what="stream")
    mean, rstd = bref.following(cpu(b.x), 2)[2:]
    want = torch.cat((mean, rstd), 1)
    assert ((b.stats.cpu().double() - want).abs() <= 2.0 ** -23 * want.abs() + 2.0 ** -40).all()


def test_prompt_then_tokens():
    """A sequence appended and attended in chunks, then token by token, in place in its projection, sees what one pass
    over it sees: places run on, and padded tokens between are not written."""
    heads, kv_heads, dim, page, n = 8, 2, 64, 16, 75
    q, W = heads * dim, kv_heads * dim
    qkv = ref.bf16((n, q + 2 * W), 1)
    place = torch.arange(n, dtype=torch.int32)[:, None] + 100000
    turn = (place, kq.rope_freqs((dim,), 1e6, "cpu"), (dim,), True)
    table = torch.randperm(9, generator=torch.Generator().manual_seed(4))[:5].reshape(1, 5).to(torch.int32)
    cache = kq.alloc_cache(9 * page, W, DEV)
    slots = ref.slots_of(table, 0, n, page, 9 * page).to(torch.int32)
    x = qkv.to(DEV)
    out, lse = torch.empty((n, q), dtype=torch.bfloat16, device=DEV), torch.empty((n, heads), device=DEV)
    freqs, at = turn[1].to(DEV), 0
    for m in [40, 27] + [1] * 8:
        pad = 3  # rows behind the chunk, without a slot
        rows = torch.cat((x[at:at + m], torch.full((pad, x.shape[1]), float("nan"), dtype=torch.bfloat16, device=DEV)))
        sl = torch.cat((slots[at:at + m], torch.full((pad,), -1, dtype=torch.int32))).to(DEV)
        pos = torch.cat((place[at:at + m], torch.zeros((pad, 1), dtype=torch.int32))).to(DEV)
        kq.kq_cache_write_rope(rows[:, q:q + W], rows[:, q + W:], sl, *cache, kv_heads,
                               rotation=kq.Rotation(pos, freqs, (dim,), True), Q=rows[:, :q], q_out=rows[:, :q], q_heads=heads)
        lens = torch.tensor([at + m], dtype=torch.int32, device=DEV)
        kq.kq_attention_mx(rows[:m, :q], *cache, lens, out[at:at + m], heads, kv_heads, page_size=page,
                           page_table=table.to(DEV), causal=True, lse=lse[at:at + m])
        at += m
    torch.cuda.synchronize()
    turned = bref.rounded(bref.rope(qkv[:, :q], heads, turn)[0]).to(torch.bfloat16)
    keys = bref.rounded(bref.rope(qkv[:, q:q + W], kv_heads, turn)[0]).to(torch.bfloat16)
    bref.check_codes(cache[0].cpu()[slots.long()], cache[1].cpu()[slots.long()], keys)
    lens = torch.tensor([n], dtype=torch.int32)
    ref.check_attention(out, lse, ref.attention(turned, [t.cpu() for t in cache], lens, table, page, heads, kv_heads,
                                                [0, n], causal=True))


class Step:
    """The decode step of a batch: one token each, far into its context, a wide residual stream."""

    def __init__(self, seed, batch=5, heads=16, kv_heads=2, dim=128, d=2240):
        self.heads, self.kv_heads, W = heads, kv_heads, kv_heads * dim
        self.q, self.W = heads * dim, W
        self.qkv = ref.bf16((batch, self.q + 2 * W), seed).to(DEV)
        self.start, self.y = ref.bf16((batch, d), seed + 1).to(DEV), ref.bf16((batch, d), seed + 2).to(DEV)
        self.x, self.qo = torch.empty_like(self.start), torch.empty((batch, self.q), dtype=torch.bfloat16, device=DEV)
        self.codes = kq.alloc_outputs(self.x)
        self.cache = kq.alloc_cache(64, W, DEV)
        g = torch.Generator().manual_seed(seed)
        self.slots = torch.randperm(64, generator=g)[:batch].to(torch.int32).to(DEV)
        place = torch.randint(0, 10 ** 6, (batch, 1), generator=g).to(torch.int32).to(DEV)
        self.rotation = kq.Rotation(place, kq.rope_freqs((dim,), 1e6, DEV), (dim,), True)

    def run(self, **kw):
        q, W = self.q, self.W
        kq.kq_cache_write_rope(self.qkv[:, q:q + W], self.qkv[:, q + W:], self.slots, *self.cache, self.kv_heads,
                               rotation=self.rotation, norm=kq.KQ_NORM_RMS, Q=self.qkv[:, :q], q_out=self.qo,
                               q_heads=self.heads, **kw)
        kq.kq_rope(self.qo, self.qo, self.heads, norm=kq.KQ_NORM_RMS, **kw)  # a norm alone, in place
        kq.kq_residual_norm(self.start, self.y, self.x, post=kq.KQ_NORM_RMS, pre=kq.KQ_NORM_RMS, out_codes=self.codes[0],
                            out_scales=self.codes[1], **kw)

    def outputs(self):
        return [t.clone() for t in (self.x, self.qo, *self.cache, *self.codes)]


def same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


def clear(thing):
    for t in (thing.x, *thing.cache, *(thing.codes if isinstance(thing.codes, tuple) else ())):
        t.zero_()


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


@pytest.mark.parametrize("kind", [Block, Step])
def test_captured_and_replayed(kind):
    """Two captured graphs replayed in turn, with eager calls of the same kind between; the rotation's host struct is read
    at capture."""
    a, b, other = kind(11), kind(12), kind(13)
    want = []
    for t in (a, b, other):
        t.run()
        torch.cuda.synchronize()
        want.append(t.outputs())
    ga, gb = capture(a), capture(b)
    for _ in range(3):
        for t in (a, b):
            clear(t)
        ga.replay()
        gb.replay()
        other.run()
        torch.cuda.synchronize()
        assert same(a.outputs(), want[0]) and same(b.outputs(), want[1]) and same(other.outputs(), want[2])


def test_a_stream_that_is_not_the_current_one():
    things = [Step(20 + i) for i in range(4)]
    want = []
    for t in things:
        t.run()
        torch.cuda.synchronize()
        want.append(t.outputs())
        clear(t)
    streams = [torch.cuda.Stream() for _ in things]
    torch.cuda.synchronize()
    for i, (t, s) in enumerate(zip(things, streams)):
        for _ in range(3):
            t.run(stream=(s, s.cuda_stream, 0)[i % 3])
    torch.cuda.synchronize()
    assert all(same(t.outputs(), w) for t, w in zip(things, want))


def test_threads_on_their_own_streams():
    things = [Step(30), Block(31), Step(32), Block(33)]
    want = []
    for t in things:
        t.run()
        torch.cuda.synchronize()
        want.append(t.outputs())
        clear(t)
    torch.cuda.synchronize()
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


def test_refusals_with_tensors():
    """The binding on tensors that do not fit; what the library itself refuses comes as its status."""
    t = Step(40)
    x, q = t.start, t.qkv
    bad = [lambda: kq.kq_rope(q, q[:, :8], 2), lambda: kq.kq_rope(q.float(), q, 2), lambda: kq.kq_rope(q.t(), q.t(), 1),
           lambda: kq.kq_rope(q, q, 20, rotation=kq.Rotation(t.rotation.positions[:2], *t.rotation[1:])),
           lambda: kq.kq_rope(q, q, 20, rotation=kq.Rotation(t.rotation.positions.long(), *t.rotation[1:])),
           lambda: kq.kq_rope(q, q, 20, rotation=kq.Rotation(t.rotation.positions, t.rotation.freqs.float(), (128,))),
           lambda: kq.kq_rope(q, q, 20, rotation=kq.Rotation(t.rotation.positions, t.rotation.freqs, (64,))),
           lambda: kq.kq_rope(q, q, 20, norm=1, weight=x[0].float()),
           lambda: kq.kq_cache_write_rope(q[:, :256], None, t.slots, *t.cache, 2, Q=q[:, 256:512]),
           lambda: kq.kq_cache_write_rope(q[:, :256], None, t.slots, *t.cache, 2, Q=q[:, 256:512], q_out=x, q_heads=2),
           lambda: kq.kq_cache_write_rope(q[:, :256], None, t.slots[:2], *t.cache, 2),
           lambda: kq.kq_cache_write_rope(q[:, :128], None, t.slots, *t.cache, 1),
           lambda: kq.kq_residual_norm(x, t.y, t.x[:2]), lambda: kq.kq_residual_norm(x, t.y, t.x, gate=x.float()),
           lambda: kq.kq_residual_norm(x, t.y, t.x, gate=x.float(), tokens_per_sample=0),
           lambda: kq.kq_residual_norm(x, t.y, t.x, post=1, post_weight=x[0]),
           lambda: kq.kq_residual_norm(x, t.y, t.x, pre=1, row_stats=x.float())]
    for call in bad:
        with pytest.raises((ValueError, TypeError, AttributeError)):
            call()
    for status, call in ((4, lambda: kq.kq_rope(q, q, 20, norm=kq.KQ_NORM_LAYER)),
                         (6, lambda: kq.kq_residual_norm(x, t.y, t.y)), (4, lambda: kq.kq_residual_norm(x, None, t.x)),
                         (2, lambda: kq.kq_rope(q[:, :36], t.qo[:, :36], 3)), (3, lambda: kq.kq_rope(q[:, 4:36], t.qo[:, :32], 1)),
                         (1, lambda: kq.kq_residual_norm(x, t.y, None))):
        with pytest.raises(kq.KQError) as e:
            call()
        assert e.value.status == status


def written(thing):
    """Everything that a run writes."""
    if isinstance(thing, Step):
        return [thing.x, thing.qo, *thing.cache, *thing.codes]
    return [thing.x, thing.stats, thing.q, thing.att, thing.h1, thing.qkv, thing.y1, thing.h, thing.y2, thing.lse, *thing.cache,
            *(t for pair in thing.codes.values() for t in pair)]


def poison(thing):
    for t in written(thing):
        t.view(torch.uint8).fill_(0xA5)


def expected(thing):
    """What a run leaves behind in poisoned buffers (slots without a token keep the poison)."""
    poison(thing)
    thing.run()
    torch.cuda.synchronize()
    return [t.clone() for t in written(thing)]


@pytest.mark.parametrize("kind", [Block, Step])
def test_replays_write_everything(kind):
    a, b = kind(51), kind(52)
    want = [expected(t) for t in (a, b)]
    ga, gb = capture(a), capture(b)
    for _ in range(3):
        poison(a)
        poison(b)
        ga.replay()
        gb.replay()
        torch.cuda.synchronize()
        assert same(written(a), want[0]) and same(written(b), want[1])


def test_threads_write_everything():
    things = [Step(60), Block(61), Step(62), Block(63)]
    want = [expected(t) for t in things]
    streams, got = [torch.cuda.Stream() for _ in things], [[] for _ in things]
    errors = []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(4):
                    poison(things[i])
                    things[i].run()
                    got[i].append([t.clone() for t in written(things[i])])
        except Exception as e:  # reported below, in the main thread
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(things))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert all(same(g, want[i]) for i in range(len(things)) for g in got[i])


@pytest.mark.parametrize("given", ["stream", "address", "default"])
def test_the_stream_given_orders_the_calls(given):
    """The inputs come to be on the stream given, behind long work, and are not there yet when the calls are made from
    another current stream; what the calls wrote is copied on the stream given."""
    t = Step(70)
    want = expected(t)
    inputs = (t.qkv, t.start, t.y)
    good = [x.clone() for x in inputs]
    m = torch.randn((8192, 8192), device=DEV)
    out = torch.empty_like(m)
    s = torch.cuda.default_stream() if given == "default" else torch.cuda.Stream()
    other = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.mm(m, m, out=out)
    poison(t)
    for x in inputs:
        x.fill_(float("nan"))
    torch.cuda.synchronize()
    ready = torch.cuda.Event()
    with torch.cuda.stream(s):
        for _ in range(12):
            torch.mm(m, m, out=out)
        for x, g in zip(inputs, good):
            x.copy_(g)
        ready.record()
    with torch.cuda.stream(other):
        t.run(stream={"stream": s, "address": s.cuda_stream, "default": 0}[given])
    early = not ready.query()
    with torch.cuda.stream(s):
        got = [x.clone() for x in written(t)]
    torch.cuda.synchronize()
    assert early, "the work in front was over too soon for this test to say anything"
    assert same(got, want)
