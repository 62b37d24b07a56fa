"""The write into a latent cache and the attention of whole prompts in the expanded form, against their definitions in 64
bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_11_gb300 as pkv
from tests.drafted_helpers import D, LATENT, ROPE, ROW, SENTINEL, U, attend64
from tests.fp8_helpers import cos_sin_table

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


# ------------------------------------------------------------------ the write
class Write:
    """Tokens of a call: runs of (first position, tokens), padding rows (slot -1) among them where `pads` says."""

    def __init__(self, seed, spans, heads, bs, dtype, inter=False, norm=True, rot=True, pads=(), fused=True, rows_at=400):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)
        self.dtype, self.inter, self.heads, self.bs = dtype, inter, heads, bs
        slots, pos, nb = [], [], 3
        blocks = sum((p + n - 1) // bs - p // bs + 1 for p, n in spans) + nb
        perm = torch.randperm(blocks, generator=g).tolist()
        for p, n in spans:
            mine = {}
            for t in range(p, p + n):
                if t // bs not in mine:
                    mine[t // bs] = perm.pop()
                slots.append(mine[t // bs] * bs + t % bs)
                pos.append(t)
        for at in pads:
            slots.insert(at, -1 - at)
            pos.insert(at, 1 << 40)       # not read
        n = len(slots)
        self.n = n
        self.slots, self.pos = torch.tensor(slots, dtype=torch.int64), torch.tensor(pos, dtype=torch.int64)
        wide = rnd(n, heads * 192 + ROW + 8) if fused else rnd(n, heads * 192 + ROW)
        wide = (wide * 2).to(dtype).cuda()
        self.q = wide[:, :heads * 192].reshape(n, heads, 192)[:, :, D:] if not fused else \
            wide[:, :heads * 192].unflatten(1, (heads, 192))[:, :, D:] if heads else None
        self.kv = wide[:, heads * 192:heads * 192 + ROW]
        if not heads:
            self.q = None
        self.table = cos_sin_table(rows_at, ROPE).cuda() if rot else None
        self.norm = (1 + 0.2 * rnd(LATENT)).to(dtype).cuda() if norm else None
        self.cache = rnd(blocks, bs, ROW).to(dtype).cuda()
        self.before = self.cache.clone()
        self.eps = 1e-5

    def call(self, **kw):
        kw = dict(kv_norm=self.norm, norm_eps=self.eps, interleaved=self.inter) | kw
        return pkv.paged_latent_append_rope(self.q, self.kv, self.pos.cuda(), self.table, self.slots.cuda(), self.cache, **kw)

    def turned(self, x, t):
        """x [..., 64] in 64 bits -> turned values and |a| + |b| of their pairs."""
        if self.table is None:
            return x, x.abs()
        row = self.table[self.pos[t]].double()
        c, s = row[:32], row[32:]
        a, b = (x[..., 0::2], x[..., 1::2]) if self.inter else (x[..., :32], x[..., 32:])
        ya, yb, m = a * c - b * s, b * c + a * s, a.abs() + b.abs()
        if self.inter:
            return torch.stack([ya, yb], -1).flatten(-2), torch.stack([m, m], -1).flatten(-2)
        return torch.cat([ya, yb], -1), torch.cat([m, m], -1)

    def close(self, got, y, mag):
        """Within the rounding of y and 1.25 * 2^-20 of mag: the sum of 512 squares in 32 bits, a root, a division and two
        products (some 30 roundings of 2^-24), and three roundings of the turn."""
        off = (got.double() - y).abs()
        tiny = 2.0 ** -25 if self.dtype == FP else 1e-40
        assert (off <= U[self.dtype] * y.abs() + 32 * 2.0 ** -24 * mag + tiny).all(), float(off.max())

    def check(self, q_out, kv_out=None, bad=()):
        expect = self.before.clone()
        kv = self.kv.double()
        for t in range(self.n):
            slot = int(self.slots[t])
            if slot < 0 or t in bad:
                continue
            c = kv[t, :LATENT]
            if self.norm is not None:
                c = c / torch.sqrt((c * c).mean() + self.eps) * self.norm.double()
            r, m = self.turned(kv[t, LATENT:], t)
            got = self.cache[slot // self.bs, slot % self.bs]
            self.close(got, torch.cat([c, r]), torch.cat([c.abs(), m]))
            if self.norm is None:
                assert torch.equal(got[:LATENT], self.kv[t, :LATENT])
            expect[slot // self.bs, slot % self.bs] = got
            if kv_out is not None:
                assert torch.equal(kv_out[t], got)
            if self.q is not None:
                y, m = self.turned(self.q_before[t].double() if hasattr(self, "q_before") else self.q[t].double(), t)
                self.close(q_out[t], y, m)
        assert torch.equal(self.cache, expect)      # and nothing else was written


SPANS = [[(0, 1)], [(0, 16), (5, 1), (31, 2)], [(3, 40), (0, 33), (15, 1)], [(7, 150)]]


@pytest.mark.parametrize("spans", range(len(SPANS)))
@pytest.mark.parametrize("heads,bs,dtype,inter,norm,rot", [
    (16, 16, BF, True, True, True), (128, 32, BF, False, True, True), (1, 16, FP, True, False, True),
    (5, 32, FP, False, True, True), (0, 16, BF, False, True, True), (17, 16, FP, False, True, False), (40, 7, BF, True, True, True)])
def test_writes(gpu, heads, bs, dtype, inter, norm, rot, spans):
    w = Write(spans + heads, SPANS[spans], heads, bs, dtype, inter, norm, rot)
    kv_out = torch.full((w.n, ROW), SENTINEL, dtype=dtype, device=gpu)
    q = w.call(kv_out=kv_out)
    assert pkv.check_device_error() == 0
    w.check(q, kv_out)


def test_outputs_in_wider_rows_and_in_place(gpu):
    w = Write(1, [(3, 20)], 8, 16, BF)
    wide = torch.full((20, 8, ROW), SENTINEL, dtype=BF, device=gpu)
    q = w.call(q_out=wide[:, :, LATENT:])
    assert pkv.check_device_error() == 0
    assert q.data_ptr() == wide[:, :, LATENT:].data_ptr() and (wide[:, :, :LATENT] == SENTINEL).all()
    w.check(q)
    w = Write(1, [(3, 20)], 8, 16, BF)
    w.q_before = w.q.clone()
    again = w.call(q_out=w.q)
    assert torch.equal(again, q)
    w.check(again)
    # rows of the latent projection alone, normed in place
    w = Write(2, [(0, 30)], 0, 16, FP)
    rows = w.kv.contiguous()
    held = rows.clone()
    w.kv = rows
    w.call(kv_out=rows)
    w.kv = held
    w.check(None, rows)


def test_padding_keeps_its_rows(gpu):
    w = Write(3, [(0, 9), (4, 20)], 6, 16, BF, pads=(0, 5, 6, 20, 33))
    q_out = torch.full((w.n, 6, ROPE), SENTINEL, dtype=BF, device=gpu)
    kv_out = torch.full((w.n, ROW), SENTINEL, dtype=BF, device=gpu)
    w.call(q_out=q_out, kv_out=kv_out)
    assert pkv.check_device_error() == 0
    w.check(q_out, kv_out)
    pad = w.slots < 0
    assert (q_out[pad] == SENTINEL).all() and (kv_out[pad] == SENTINEL).all()
    w = Write(4, [], 3, 16, BF)
    assert w.call().shape == (0, 3, ROPE)


def test_bad_slots_and_positions(gpu):
    for what, code in (("slot", 1), ("pos", 8), ("neg", 8)):
        w = Write(5, [(0, 12)], 4, 16, BF)
        if what == "slot":
            w.slots[7] = w.cache.shape[0] * 16
        else:
            w.pos[7] = 400 if what == "pos" else -1
        kv_out = torch.full((w.n, ROW), SENTINEL, dtype=BF, device=gpu)
        q = w.call(kv_out=kv_out)
        assert pkv.check_device_error() == code
        w.check(q, kv_out, bad=(7,))
        assert (q[7] == 0).all() and (kv_out[7] == 0).all()


def test_rows_that_are_not_finite_or_zero(gpu):
    """Each row is its own: the others are as without it."""
    w = Write(6, [(0, 5)], 4, 16, BF)
    w.kv[2, 3], w.kv[3] = float("inf"), 0.0
    q = w.call()
    assert pkv.check_device_error() == 0
    s = [int(x) for x in w.slots]
    assert torch.isnan(w.cache[s[2] // 16, s[2] % 16, 3]) and (w.cache[s[3] // 16, s[3] % 16] == 0).all()
    w.before[s[2] // 16, s[2] % 16] = w.cache[s[2] // 16, s[2] % 16]
    got = w.cache.clone()
    w.cache.nan_to_num_(), w.before.nan_to_num_()
    w.check(q, bad=(2,))
    assert not torch.isnan(got).all()


# ------------------------------------------------------------------ prompts
class Prompts:
    """Packed prompts of (queries, keys).  extra: tokens behind the last prompt, of queries and keys, that are NaN."""

    def __init__(self, seed, seqs, heads, dtype, extra=0, slices=False, scale=None, gap=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.seqs, self.heads, self.dtype = seqs, heads, dtype
        self.scale = 192 ** -0.5 if scale is None else scale
        qs, ks = [gap], [gap]
        for n, m in seqs:
            qs.append(qs[-1] + n)
            ks.append(ks[-1] + m)
        self.qs_list, self.ks_list = qs, ks
        self.qs, self.ks = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (qs, ks))
        Tq, Tk = qs[-1] + extra, ks[-1] + extra
        if slices:      # heads and tokens apart
            self.q = rnd(Tq, heads + 2, 200).to(dtype)[:, 1:heads + 1, 8:]
            self.kv = rnd(Tk, heads + 1, 264).to(dtype)[:, :heads, :256]
            self.k_rope = rnd(Tk, ROW).to(dtype)[:, LATENT:]
        else:
            self.q, self.kv, self.k_rope = (x.to(dtype) for x in (rnd(Tq, heads, 192), rnd(Tk, heads, 256), rnd(Tk, ROPE)))
        for x, end in ((self.q, qs[-1]), (self.kv, ks[-1]), (self.k_rope, ks[-1])):
            x[end:], x[:gap] = float("nan"), float("nan")
        self.out = torch.full((Tq, heads, D), SENTINEL, dtype=dtype, device="cuda")

    def call(self, **kw):
        kw = dict(max_query_len=max([n for n, _ in self.seqs] + [0]), out=self.out) | kw
        return pkv.latent_attention_prefill(self.q, self.kv, self.k_rope, self.qs, self.ks, self.scale, **kw)

    def expected(self, s):
        n, m = self.seqs[s]
        a, b = self.qs_list[s], self.ks_list[s]
        q = self.q[a:a + n].double().transpose(0, 1)
        kv = self.kv[b:b + m].double().transpose(0, 1)
        k = torch.cat([kv[..., :D], self.k_rope[b:b + m].double()[None].expand(self.heads, -1, -1)], dim=-1)
        i = torch.arange(n, device="cuda")[:, None]
        seen = torch.arange(m, device="cuda")[None, :] <= i + (m - n)
        y, bound = attend64(q, k, kv[..., D:], seen, self.scale, self.dtype)
        return y.transpose(0, 1), bound.transpose(0, 1)

    def check(self, out=None, only=None, zeros=()):
        out = self.out if out is None else out
        for s in range(len(self.seqs)) if only is None else only:
            n, m = self.seqs[s]
            got = out[self.qs_list[s]:self.qs_list[s] + n].double()
            if s in zeros:
                assert (got == 0).all()
                continue
            y, b = self.expected(s)
            off = (got - y).abs()
            assert (off <= b).all(), (s, n, m, int((~(off <= b)).sum()), float((off / b).nan_to_num(1e30).max()))
        assert (out[self.qs_list[-1]:] == SENTINEL).all() and (out[:self.qs_list[0]] == SENTINEL).all()


def run(p, expect=0, **kw):
    out = p.call(**kw)
    assert pkv.check_device_error() == expect
    return out


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n", [1, 2, 63, 64, 127, 128, 129, 200, 255, 256, 257, 383, 384, 385, 512, 700, 1025])
def test_prompt_lengths(gpu, n, dtype):
    p = Prompts(n, [(n, n)], 3, dtype, extra=2)
    run(p)
    p.check()


@pytest.mark.parametrize("prefix", [1, 63, 64, 128, 129, 500, 1000])
@pytest.mark.parametrize("n", [1, 100, 128, 300, 513])
def test_prompts_behind_a_prefix(gpu, n, prefix):
    p = Prompts(n + prefix, [(n, n + prefix)], 2, BF, extra=1)
    run(p)
    p.check()


@pytest.mark.parametrize("heads,slices", [(1, False), (16, True), (40, False), (7, True)])
def test_ragged_prompts(gpu, heads, slices):
    seqs = [(5, 5), (0, 0), (300, 300), (1, 1), (0, 40), (129, 400), (257, 257), (64, 64)]
    for dtype in (BF, FP):
        p = Prompts(heads, seqs, heads, dtype, extra=3, slices=slices, gap=4)
        run(p)
        p.check()
        first = p.out.clone()
        run(p, max_query_len=None)
        assert torch.equal(p.out, first)


def test_queries_without_keys(gpu):
    """Fewer keys than queries: the first queries attend nothing."""
    for n, m in ((10, 4), (300, 5), (300, 290), (400, 130), (50, 0), (700, 0)):
        p = Prompts(n, [(n, m), (20, 20)], 2, BF)
        run(p)
        p.check()
        assert (p.out[:n - m] == 0).all()
    p = Prompts(1, [(5, 0)], 2, BF)      # no keys at all in the call
    run(p)
    assert (p.out == 0).all()


@pytest.mark.parametrize("scale", [0.0, -0.05, 2.0])
def test_prompt_scales(gpu, scale):
    p = Prompts(3, [(300, 300)], 2, BF, scale=scale)
    run(p)
    p.check()


def test_prompt_scores_that_rise(gpu):
    for sign in (1, -1):
        p = Prompts(4, [(900, 900)], 2, BF)
        p.q[..., 0] = 8.0
        p.kv[:, :, 0] = (sign * torch.arange(900, device=gpu)[:, None] / 900 * 60).to(BF)
        run(p)
        p.check()


@pytest.mark.parametrize("what", [float("inf"), float("-inf"), float("nan")])
def test_prompt_values_that_are_not_finite(gpu, what):
    """A key's value that is not finite spoils the queries from its own on, in its dims, and none before."""
    for n, m, at in ((9, 9, 4), (300, 300, 140), (300, 300, 10), (300, 300, 299), (600, 900, 700), (130, 130, 129), (257, 257, 256)):
        p = Prompts(5, [(n, m), (40, 40)], 2, BF)
        p.kv[at, 1, D + 77] = what
        run(p)
        got = p.out.clone()
        p.kv[at, 1, D + 77] = 0.5
        first = max(0, at - (m - n))    # first query that attends it
        y, b = p.expected(0)
        ok = (got[:n].double() - y).abs() <= b
        assert ok[:first].all() and ok[:, 0].all()
        assert not torch.isfinite(got[first:n, 1, 77]).any()
        # beside it nothing is spoiled (its own weight is the same whatever the value)
        ok[first:, 1, 77] = True
        assert ok.all()
        p.out.copy_(got)
        p.check(only=[1])


def test_prompt_keys_that_are_not_finite(gpu):
    p = Prompts(6, [(300, 300)], 2, BF)
    y, b = p.expected(0)
    p.k_rope[200, 3] = float("nan")
    run(p)
    assert ((p.out[:200].double() - y[:200]).abs() <= b[:200]).all() and torch.isnan(p.out[200:]).all()


def test_prompt_bad_metadata(gpu):
    make = lambda: Prompts(7, [(100, 100), (300, 310), (40, 40)], 2, BF, extra=2)
    p = make()
    p.ks[2] = 1 << 30
    run(p, expect=10)
    p.check(zeros=[1, 2])
    p = make()
    run(p, expect=10, max_query_len=299)
    p.check(zeros=[1])
    p = make()
    p.qs[1] = -1
    run(p, expect=10)
    assert (p.out[:400] == SENTINEL).all()
    p.check(only=[2])
    p = make()
    p.qs[3] = 500000
    run(p, expect=10)
    assert (p.out[400:] == SENTINEL).all()
    p.check(only=[0, 1])


MANY = [(5, 5), (0, 0), (300, 300), (1, 1), (0, 40), (129, 400), (700, 200), (257, 257), (3, 0), (64, 64), (900, 1500), (256, 256)]


@pytest.mark.parametrize("heads,dtype,slices", [(48, BF, False), (33, FP, True), (128, BF, True)])
def test_more_prompts_than_ctas(gpu, heads, dtype, slices):
    """Grids of many times the SMs, most of whose places are empty or short, with and without a bound of the lengths."""
    p = Prompts(9, MANY, heads, dtype, extra=3, slices=slices, gap=4)
    p.check(run(p))
    p.out.fill_(SENTINEL)
    p.check(run(p, max_query_len=None))


def test_more_prompts_than_ctas_with_bad_metadata(gpu):
    make = lambda: Prompts(10, MANY, 48, BF, extra=2)
    p = make()
    run(p, expect=10, max_query_len=299)
    p.check(zeros=[2, 6, 10])
    p = make()
    p.ks[9] = -5
    run(p, expect=10)
    p.check(zeros=[8, 9])
    p = make()
    p.qs[5] = 1 << 30
    run(p, expect=10)
    p.check(only=[0, 1, 2, 3, 6, 7, 8, 9, 10, 11])
    assert (p.out[p.qs_list[5]:p.qs_list[6]] == SENTINEL).all()


def test_many_prompts_at_once(gpu):
    """Two streams and a graph whose grids are larger than the SMs."""
    ps = [Prompts(11 + i, [(700 + i, 800), (40, 40), (600, 600)], 64, BF) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(4):
        for p, s in zip(ps, streams):
            p.call(stream=s)
    torch.cuda.synchronize()
    assert pkv.check_device_error() == 0
    for p in ps:
        p.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for p in ps:
            p.call()
    for p in ps:
        p.q.copy_(torch.randn_like(p.q))
        p.out.fill_(SENTINEL)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert pkv.check_device_error() == 0
    for p in ps:
        p.check()


def test_prompts_on_streams_and_in_graphs(gpu):
    ps = [Prompts(8 + i, [(500 + i, 600), (40, 40)], 4, BF) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(3):
        for p, s in zip(ps, streams):
            p.call(stream=s)
    torch.cuda.synchronize()
    for p in ps:
        p.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for p in ps:
            p.call()
    for p in ps:
        p.q.copy_(torch.randn_like(p.q))
        p.out.fill_(SENTINEL)
    g.replay()
    assert pkv.check_device_error() == 0
    for p in ps:
        p.check()


# ------------------------------------------------------------------ together
def test_a_prompt_and_its_decode_steps(gpu):
    """Prompts through the write and the expanded form, then a decode step and a tree of drafted tokens through the absorbed
    form: a layer of latent attention with its expansions, against the expanded form in 64 bits over the cached rows."""
    H, bs, scale = 8, 16, 192 ** -0.5
    g = torch.Generator(device=gpu).manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=g, device=gpu)
    w = (rnd(H, 256, LATENT) * LATENT ** -0.5).to(BF)     # expansion of a latent: a head's key, then its value
    lens, drafts = [70, 5, 300], [4, 1, 7]
    table = cos_sin_table(512, ROPE).cuda()
    norm = (1 + 0.1 * rnd(LATENT)).to(BF)
    nblk = [-(-(L + n) // bs) for L, n in zip(lens, drafts)]
    perm = torch.randperm(sum(nblk), generator=g, device=gpu).int()
    tables = torch.full((3, max(nblk)), -1, dtype=torch.int32, device=gpu)
    at = 0
    for s, n in enumerate(nblk):
        tables[s, :n] = perm[at:at + n]
        at += n
    cache = torch.full((sum(nblk), bs, ROW), float("nan"), dtype=BF, device=gpu)

    def tokens(firsts, counts):
        pos = torch.cat([torch.arange(p, p + n, device=gpu) for p, n in zip(firsts, counts)])
        seq = torch.repeat_interleave(torch.arange(3, device=gpu), torch.tensor(counts, device=gpu))
        starts = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=gpu)
        return pos, tables[seq, pos // bs].long() * bs + pos % bs, starts

    def write(firsts, counts):
        T = sum(counts)
        q, kv = rnd(T, H, 192).to(BF), (rnd(T, ROW) * 2).to(BF)
        pos, slots, starts = tokens(firsts, counts)
        rows = torch.empty(T, ROW, dtype=BF, device=gpu)
        pkv.paged_latent_append_rope(q[:, :, D:], kv, pos, table, slots, cache, kv_norm=norm, q_out=q[:, :, D:], kv_out=rows)
        return q, rows, starts

    def reference(q, s, L, seen):
        t = torch.arange(L, device=gpu)
        r = cache[tables[s, t // bs].long(), t % bs].double()
        kv = torch.einsum("hdc,tc->htd", w.double(), r[:, :LATENT])
        k = torch.cat([kv[..., :D], r[None, :, LATENT:].expand(H, -1, -1)], dim=-1)
        return attend64(q.double().transpose(0, 1), k, kv[..., D:], seen, scale, BF)[0].transpose(0, 1)

    # prompts: the expanded keys and values are rounded to bf16 (2^-8 each); so are the absorbed queries and outputs below.
    # A score of sd 1.8 moves by some 2^-8 of its size, an output by some 3 roundings of 2^-8: 0.05 of the largest value (4.5)
    q, rows, starts = write([0, 0, 0], lens)
    kv = torch.einsum("tc,hdc->thd", rows[:, :LATENT].float(), w.float()).to(BF)
    out = pkv.latent_attention_prefill(q, kv, rows[:, LATENT:], starts, starts, scale, max_query_len=max(lens))
    assert pkv.check_device_error() == 0
    for s, L in enumerate(lens):
        i = torch.arange(L, device=gpu)
        a = int(starts[s])
        assert (out[a:a + L].double() - reference(q[a:a + L], s, L, i[None, :] <= i[:, None])).abs().max() < 0.05

    def absorbed(firsts, counts, masks):
        q, _, starts = write(firsts, counts)
        qa = torch.cat([torch.einsum("thd,hdc->thc", q[..., :D].float(), w[:, :D].float()).to(BF), q[..., D:]], dim=-1)
        total = torch.tensor([p + n for p, n in zip(firsts, counts)], dtype=torch.int32, device=gpu)
        o = pkv.paged_latent_decode(qa, cache, tables, total, scale, query_starts=starts, tree_masks=masks)
        out = torch.einsum("thc,hdc->thd", o.float(), w[:, D:].float())
        assert pkv.check_device_error() == 0
        for s, (p, n) in enumerate(zip(firsts, counts)):
            a = int(starts[s])
            i = torch.arange(n, device=gpu)
            mine = i[None, :] <= i[:, None] if masks is None else (masks[a:a + n, None] >> i[None, :]) & 1 == 1
            seen = torch.cat([torch.ones(n, p, dtype=torch.bool, device=gpu), mine], dim=1)
            assert (out[a:a + n].double() - reference(q[a:a + n], s, p + n, seen)).abs().max() < 0.05

    absorbed(lens, [1, 1, 1], None)
    from tests.drafted_helpers import tree_masks
    absorbed(lens, drafts, tree_masks(torch.Generator().manual_seed(1), drafts).to(gpu))
