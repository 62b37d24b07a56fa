"""Attention of drafted tokens over a K/V cache (paged_attention_tree) and over a latent cache (paged_latent_decode), against
its definition in 64 bits.  Every place of the pools that no sequence holds is NaN."""
import pytest
import torch

import paged_kv_cache_11_gb300 as pkv
from tests.drafted_helpers import SENTINEL, Batch

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
KINDS = ["tree", "latent"]


def run(b, expect=0, **kw):
    out = b.call(**kw)
    assert pkv.check_device_error() == expect
    return out


# ------------------------------------------------------------------ sizes
@pytest.mark.parametrize("n", [1, 2, 5, 31, 64])
@pytest.mark.parametrize("kind,heads,hkv", [("tree", 4, 1), ("tree", 8, 2), ("tree", 7, 7), ("tree", 24, 3),
                                            ("latent", 1, 1), ("latent", 16, 1), ("latent", 40, 1), ("latent", 128, 1)])
def test_lengths_and_heads(gpu, kind, heads, hkv, n):
    """Contexts around the tiles' and blocks' ends, from the drafted tokens alone on."""
    lens = [n, n + 1, 63 + n, 64, 65, 127, 128, 129, 200, 256, 257, 385]
    seqs = [(max(L, n), n) for L in lens]
    for bs, dtype, masks in ((16, BF, "tree"), (32, FP, "chain")):
        b = Batch(10 * n + heads + bs, seqs, heads, hkv, bs, dtype, kind, masks, extra=3)
        run(b)
        b.check()


@pytest.mark.parametrize("kind", KINDS)
def test_ragged_batches(gpu, kind):
    """Sequences of different n, some without drafted tokens, some empty."""
    seqs = [(300, 7), (0, 1), (5, 5), (1000, 0), (64, 64), (0, 4), (17, 1), (0, 0), (700, 33), (129, 64)]
    for seed, (heads, hkv) in enumerate([(32, 8), (16, 1), (64, 1)] if kind == "tree" else [(16, 1), (64, 1), (3, 1)]):
        for masks in ("tree", "chain", "random"):
            b = Batch(seed, seqs, heads, hkv, 16, BF, kind, masks, extra=5)
            run(b)
            b.check()


@pytest.mark.parametrize("kind", KINDS)
def test_one_token_a_sequence(gpu, kind):
    b = Batch(3, [(L, 1) for L in (1, 2, 16, 100, 0, 513, 2000)], 16, 2 if kind == "tree" else 1, 32, BF, kind, "chain",
              starts=False)
    run(b)
    b.check()


@pytest.mark.parametrize("kind,heads,hkv", [("tree", 8, 1), ("tree", 40, 40), ("latent", 16, 1), ("latent", 128, 1)])
def test_long_contexts_are_divided(gpu, kind, heads, hkv):
    """A few long contexts: every unit is cut between CTAs."""
    for seed, seqs in enumerate([[(20000, 3)], [(9000, 1), (40, 2), (12345, 9)], [(4097, 64)]]):
        b = Batch(seed, seqs, heads, hkv, 16 if seed else 32, FP if seed else BF, kind, "tree", width=2000)
        run(b)
        b.check()


@pytest.mark.parametrize("kind", KINDS)
def test_many_sequences(gpu, kind):
    """More sequences than a CTA has threads; many units to a CTA."""
    g = torch.Generator().manual_seed(4)
    seqs = [(int(torch.randint(0, 90, (1,), generator=g)), 1) for _ in range(1500)]
    seqs = [(L, int(L > 3) * 2 + 1) if L > 3 else (L, 1) for L, _ in seqs]
    b = Batch(5, seqs, 4, 2 if kind == "tree" else 1, 16, BF, kind, "tree")
    run(b)
    b.check(only=list(range(0, 1500, 37)) + [1499])


@pytest.mark.parametrize("kind", KINDS)
def test_more_rows_than_a_unit(gpu, kind):
    """64 drafted tokens of 64 heads to one KV head: 4096 query rows."""
    b = Batch(6, [(500, 64), (64, 64)], 64, 1, 16, FP, kind, "tree")
    run(b)
    b.check()


# ------------------------------------------------------------------ masks and values
@pytest.mark.parametrize("kind", KINDS)
def test_tokens_that_attend_nothing(gpu, kind):
    """No context before the drafted tokens and empty masks: zeros."""
    b = Batch(7, [(9, 9), (140, 9)], 16, 1, 16, BF, kind, "tree")
    b.masks[2] = 0
    b.masks[7] = ~0x1ff          # only bits behind the last drafted token
    b.masks[9] = 0               # attends its context alone
    run(b)
    b.check()
    assert (b.out[[2, 7]] == 0).all() and (b.out[9] != 0).any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [0.0, -0.07, 3.0])
def test_scales(gpu, kind, scale):
    b = Batch(8, [(300, 5), (77, 3)], 16, 1, 16, BF, kind, "tree", scale=scale)
    run(b)
    b.check()


@pytest.mark.parametrize("kind", KINDS)
def test_rising_and_falling_scores(gpu, kind):
    """Scores that rise along the context make the running maximum rise tile after tile; falling ones vanish."""
    for sign in (1, -1):
        b = Batch(9, [(1500, 4)], 16, 1, 16, BF, kind, "tree")
        q = b.q.float()
        q[..., 0] = 8.0
        b.q = q.to(BF)
        t = torch.arange(1500, device=gpu)
        blk, off = b.tables[0, t // 16].long(), t % 16
        ramp = (sign * t.float() / 1500 * 60).to(BF)
        if kind == "tree":
            b.pools[0][blk, 0, off, 0] = ramp
        else:
            b.pools[0][blk, off, 0] = ramp
        run(b)
        b.check()


@pytest.mark.parametrize("kind,heads", [("tree", 4), ("tree", 32), ("latent", 16), ("latent", 64)])
@pytest.mark.parametrize("what", [float("inf"), float("-inf"), float("nan")])
def test_values_that_are_not_finite(gpu, kind, heads, what):
    """A drafted token whose value is not finite spoils the tokens that descend from it in those dims, and no other."""
    for L, n in ((9, 9), (150, 9), (135, 9), (3000, 9)):
        b = Batch(11, [(L, n), (50, 3)], heads, 1, 16, BF, kind, "tree")
        pos, dim = L - n + 2, 5     # the third drafted token
        blk, off = int(b.tables[0, pos // 16]), pos % 16
        b.masks[2] = b.masks[2] | 4
        attends = [bool(int(b.masks[i]) >> 2 & 1) for i in range(n)]
        assert any(attends) and not all(attends)
        pool = b.pools[-1]
        at = (blk, 0, off, dim) if kind == "tree" else (blk, off, dim)
        held = pool[at].clone()
        pool[at] = what             # (of a latent cache the value is a part of the key: its score is not finite either)
        run(b)
        got = b.out.clone()
        pool[at] = held
        for i in range(n):
            y, bound = b.expected(0)
            y, bound = y[i], bound[i]
            x = got[i].double()
            if attends[i]:
                if kind == "tree":
                    assert not torch.isfinite(x[:, dim]).any()
                    rest = torch.arange(x.shape[1], device=gpu) != dim
                    assert ((x - y).abs() <= bound)[:, rest].all()
                else:
                    # a score of -inf (or NaN, +inf) by the sign of the query's value
                    assert not torch.isfinite(x[:, dim]).all()
            else:
                assert ((x - y).abs() <= bound).all(), (L, i)
        b.out.copy_(got)
        b.check(only=[1])


@pytest.mark.parametrize("kind", KINDS)
def test_keys_and_queries_that_are_not_finite(gpu, kind):
    """Keys of tokens that are not attended do not matter; a query that is not finite spoils its own row alone."""
    b = Batch(12, [(200, 6)], 16, 1, 16, BF, kind, "tree")
    pos = 200 - 6 + 3
    for i in range(6):
        if i != 3:
            b.masks[i] = b.masks[i] & ~8
    b.masks[3] = b.masks[3] | 8
    at = (int(b.tables[0, pos // 16]), 0, pos % 16) if kind == "tree" else (int(b.tables[0, pos // 16]), pos % 16)
    held = b.pools[0][at].clone()
    b.pools[0][at] = float("nan")
    run(b)
    got = b.out.clone()
    b.pools[0][at] = held
    y, bound = b.expected(0)
    keep = [i for i in range(6) if i != 3]
    assert ((got.double() - y).abs() <= bound)[keep].all() and not torch.isfinite(got[3]).any()
    b.q[1, 3] = float("nan")
    run(b)
    off = (b.out.double() - y).abs() <= bound
    off[1, 3] = True
    assert off.all() and torch.isnan(b.out[1, 3]).all()


@pytest.mark.parametrize("kind,heads", [("tree", 4), ("tree", 64), ("latent", 16), ("latent", 128)])
def test_what_is_not_finite_in_divided_contexts(gpu, kind, heads):
    """Contexts long enough to be divided: what spoils one part spoils the row, also where nothing else in that part counts."""
    n = 3
    for L in (3000, 40000):
        b = Batch(30, [(L, n), (50, 2)], heads, 1, 16, BF, kind, "tree")
        y, bound = b.expected(0)
        held = b.q[1, 3].clone()
        b.q[1, 3] = float("nan")
        run(b)
        off = (b.out[:n].double() - y).abs() <= bound
        assert torch.isnan(b.out[1, 3]).all(), L
        off[1, 3] = True
        assert off.all(), L
        b.check(only=[1])
        b.q[1, 3] = held
        # the keys of the first half of the context, more than a part of it
        ids = b.tables[0, :L // 2 // 16].long()
        b.pools[0][ids] = float("nan")
        run(b)
        assert torch.isnan(b.out[:n]).all(), L
        b.check(only=[1])


def test_a_value_of_no_weight_that_is_not_finite(gpu):
    """Where a part's weights all fall below fp32 against another's: 0 times what is not finite is not finite."""
    L, n, dim, at = 3000, 2, 9, 37
    b = Batch(31, [(L, n)], 4, 1, 16, BF, "tree", "chain")
    b.q.fill_(1.0)
    b.pools[0][b.tables[0, :1536 // 16].long()] = -20.0     # 2^-326 of the other half's weights, that are about 1
    y, bound = b.expected(0)
    b.pools[1][int(b.tables[0, at // 16]), 0, at % 16, dim] = float("inf")
    run(b)
    got = b.out.double()
    assert not torch.isfinite(got[..., dim]).any()
    ok = (got - y).abs() <= bound
    ok[..., dim] = True
    assert ok.all()


# ------------------------------------------------------------------ the order of blocks, other streams, graphs
@pytest.mark.parametrize("kind", KINDS)
def test_physical_order_does_not_matter(gpu, kind):
    b = Batch(13, [(900, 4), (333, 7)], 16, 1, 16, BF, kind, "tree")
    first = run(b).clone()
    nb = b.pools[0].shape[0]
    perm = torch.randperm(nb, device=gpu)
    for i, x in enumerate(b.pools):
        y = torch.empty_like(x)
        y[perm] = x
        b.pools[i] = y
    b.tables = torch.where(b.tables >= 0, perm.int()[b.tables.long().clamp(min=0)], -1).int()
    assert torch.equal(run(b), first)
    assert torch.equal(run(b), first)


@pytest.mark.parametrize("kind", KINDS)
def test_streams_and_outputs(gpu, kind):
    """Two calls at once on two streams, without outputs or workspaces of the caller's."""
    bs = [Batch(14 + i, [(3000 + i, 4), (100, 2)], 16, 1, 16, BF, kind, "tree") for i in range(2)]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    outs = [[b.call(out=None, stream=s) for b, s in zip(bs, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    assert pkv.check_device_error() == 0
    for row in outs:
        for b, o in zip(bs, row):
            b.check(o)


@pytest.mark.parametrize("kind", KINDS)
def test_graphs_share_a_workspace(gpu, kind):
    """Two captured calls with one workspace, replayed in turn with new inputs and lengths."""
    need = pkv.paged_attention_tree_workspace_bytes() if kind == "tree" else pkv.paged_latent_decode_workspace_bytes()
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=gpu)
    bs = [Batch(16 + i, [(2500, 3), (700, 5)], 16, 1, 16, BF, kind, "tree") for i in range(2)]
    run(bs[0], workspace=ws)
    graphs = []
    for b in bs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.call(workspace=ws)
        graphs.append(g)
    for k in range(3):
        for b in bs:
            b.q.copy_(torch.randn_like(b.q))
            b.out.fill_(SENTINEL)
            b.lens = [2500 - 600 * k, 700 - 90 * k]
            b.context_lens.copy_(torch.tensor(b.lens, dtype=torch.int32))
        for g in graphs:
            g.replay()
        assert pkv.check_device_error() == 0
        for b in bs:
            b.check()


def test_a_pool_past_4_gib(gpu):
    """Offsets past 32 bits: the sequence's blocks are the last ones of a pool of more than 2^32 bytes."""
    nb, bs = 140000, 32
    pool = torch.zeros(nb, bs, 576, dtype=BF, device=gpu)
    b = Batch(18, [(500, 3)], 16, 1, bs, BF, "latent", "tree")
    for j in range(16):
        pool[nb - 1 - j] = b.pools[0][int(b.tables[0, j])]
        b.tables[0, j] = nb - 1 - j
    b.pools = [pool]
    run(b)
    b.check()
    k = torch.zeros(70000, 8, 32, 128, dtype=BF, device=gpu)
    v = torch.zeros_like(k)
    b = Batch(19, [(500, 3)], 16, 8, 32, BF, "tree", "tree")
    for j in range(16):
        for big, small in ((k, b.pools[0]), (v, b.pools[1])):
            big[70000 - 1 - j] = small[int(b.tables[0, j])]
        b.tables[0, j] = 70000 - 1 - j
    b.pools = [k, v]
    run(b)
    b.check()


# ------------------------------------------------------------------ bad metadata
@pytest.mark.parametrize("kind", KINDS)
def test_bad_metadata(gpu, kind):
    """Reported, and the sequence's rows are zeros (or left alone where query_starts names none); others are not touched."""
    seqs = [(700, 4), (300, 3), (20, 2)]
    make = lambda: Batch(20, seqs, 16, 1, 16, BF, kind, "tree")
    b = make()
    b.tables[0, 20] = b.pools[0].shape[0]
    run(b, expect=4)
    b.check(zeros=[0])
    b = make()
    b.tables[1, 0] = -5
    run(b, expect=4)
    b.check(zeros=[1])
    for bad in (-1, 2, 44 * 16 + 1):
        b = make()
        b.context_lens[1] = bad
        run(b, expect=3)
        b.check(zeros=[1])
    b = make()
    b.starts[1] = -3                     # out of range for sequences 0 and 1
    run(b, expect=10)
    assert (b.out[:7] == SENTINEL).all()
    b.check(only=[2])
    b = make()
    b.starts[3] = 1 << 30
    run(b, expect=10)
    b.check(only=[0, 1])
    assert (b.out[7:] == SENTINEL).all()
    b = Batch(21, [(100, 2), (400, 64)], 16, 1, 16, BF, kind, "tree", extra=6)
    b.starts[2] += 1                     # 65 tokens
    run(b, expect=10)
    assert (b.out[2:67] == 0).all()
    b.starts_list[2] = 67
    b.check(only=[0])
