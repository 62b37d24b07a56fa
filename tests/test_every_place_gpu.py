"""Every position of a context or prompt counts, wherever tiles, blocks and the cuts between CTAs lie.

Keys are signs, and each query is the key of one position times 1: its score there is the key's width K, and at another
position a sum of K random signs, some sqrt(K) in size.  With all scores K apart from -K, and the others' largest (checked) at
least 40 below K, the other weights are below e^-40 n in all, far less than half a step of the output: the output is the value of
that position, bit by bit (the one weight is 2^x with |x| < 2^-16, 1 in 16 bits, and its sum's inverse is as near to 1), but for
values of exactly zero, beside which the others leave e^-40 n max |v| < 1e-12.  So a position that is left out, read twice or read from another place is seen, which sums over thousands of tokens would hide."""
import pytest
import torch

import paged_kv_cache_11_gb300 as pkv
from tests.drafted_helpers import D, LATENT, ROPE, ROW, SENTINEL
from tests.drafted_helpers import Batch
from tests.test_latent_gpu import Prompts

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def signs(gen, *shape):
    return (torch.randint(0, 2, shape, generator=gen, device="cuda", dtype=torch.int8) * 2 - 1)


def differ(a, b):
    return (a.float() - b.float()).abs() > 1e-12


def gap(keys, wanted):
    """How far below K the largest score of other positions lies, for some of the positions."""
    k = keys.float()
    s = k[wanted] @ k.t()
    s[torch.arange(len(wanted)), wanted] = -torch.inf
    return k.shape[1] - float(s.max())


class Walk(Batch):
    """A batch whose rows are each aimed at one position of their context, at other ones in each step."""

    def __init__(self, seed, seqs, heads, hkv, bs, dtype, kind):
        super().__init__(seed, seqs, heads, hkv, bs, dtype, kind, "chain", extra=2, scale=1.0, spare=1)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.keys = []      # of each sequence, [hkv, L, width]
        for s, L in enumerate(self.lens):
            k = signs(g, hkv, L, D if kind == "tree" else ROW)
            t = torch.arange(L, device="cuda")
            blk, off = self.tables[s, t // bs].long(), t % bs
            if kind == "tree":
                self.pools[0][blk, :, off] = k.transpose(0, 1).to(dtype)
            else:
                self.pools[0][blk, off] = k[0].to(dtype)
            self.keys.append(k.to(dtype))
            some = torch.randint(0, L, (64,), generator=g, device="cuda").unique()
            assert all(gap(k[h], some) >= 40 for h in range(hkv))
        self.group = heads // hkv
        self.steps = max(-(-L // (n * self.group)) for L, n in seqs if n) + 1

    def aim(self, step):
        """The position that each row is aimed at in a step: one after the other over all rows and steps; in the last step the
        drafted tokens at themselves, the last of them at all of those before it."""
        out = []
        for L, n in zip(self.lens, self.counts):
            i, g = (x.to("cuda") for x in torch.meshgrid(torch.arange(n), torch.arange(self.group), indexing="ij"))
            if step < self.steps - 1:
                at = (step * n * self.group + i * self.group + g) % (L - n + i + 1)
            else:
                at = torch.where(i == n - 1, L - 1 - g % L, L - n + i)
            out.append(at)      # [n, group]
        return out

    def step(self, step):
        """Runs it and counts the values that are not those aimed at, for each sequence."""
        aims = self.aim(step)
        for s, at in enumerate(aims):
            a, n = self.starts_list[s], self.counts[s]
            q = self.keys[s][:, at]                                      # [hkv, n, group, width]
            self.q[a:a + n] = q.transpose(0, 1).reshape(n, self.heads, -1)
        self.out.fill_(SENTINEL)
        self.call()
        wrong = []
        for s, at in enumerate(aims):
            a, n = self.starts_list[s], self.counts[s]
            blk, off = self.tables[s, at // self.bs].long(), at % self.bs
            if self.kind == "tree":
                h = torch.arange(self.hkv, device="cuda")[:, None, None]
                want = self.pools[1][blk[None], h, off[None]].transpose(0, 1).reshape(n, self.heads, D)
            else:
                want = self.pools[0][blk, off][..., :LATENT]              # [n, heads, 512]
            wrong.append(differ(self.out[a:a + n], want).any(-1).view(n, self.hkv, self.group).transpose(1, 2))
        return aims, wrong


# (kind, query heads, KV heads, [(context, drafted tokens)], block size): rows of one stream and of two, several units of rows,
# contexts of one part and of many, ends of blocks and tiles at odd places
SHAPES = [
    ("tree", 64, 1, [(20011, 64)], 32), ("tree", 32, 1, [(9001, 3), (777, 1), (2500, 5)], 16), ("tree", 20, 20, [(1500, 2)] * 4, 16),
    ("tree", 8, 8, [(40000, 31)], 16), ("tree", 24, 3, [(1283, 11)] * 9, 32), ("tree", 4, 1, [(100, 8), (37, 8), (8, 8), (65, 8)], 16),
    ("tree", 12, 2, [(129 + 16 * i, 1 + i) for i in range(40)], 16),
    ("latent", 128, 1, [(12345, 4)], 16), ("latent", 16, 1, [(9001, 3), (777, 1), (2500, 5)], 32),
    ("latent", 40, 1, [(1283, 11)] * 9, 16), ("latent", 16, 1, [(100, 1), (37, 1), (8, 1), (65, 1)], 16),
    ("latent", 64, 1, [(65 + 16 * i, 1 + i % 5) for i in range(40)], 16),
]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_every_position_of_a_context(gpu, shape, dtype):
    kind, heads, hkv, seqs, bs = SHAPES[shape]
    w = Walk(60 + shape, seqs, heads, hkv, bs, dtype, kind)
    total = torch.zeros((), dtype=torch.int64, device=gpu)
    seen = [torch.zeros(L, dtype=torch.bool, device=gpu) for L in w.lens]
    for step in range(w.steps):
        aims, wrong = w.step(step)
        for s, at in enumerate(aims):
            seen[s][at.flatten()] = True
            total += wrong[s].sum()
    assert pkv.check_device_error() == 0
    assert all(bool(x.all()) for x in seen)     # (that each was aimed at)
    assert int(total) == 0
    assert (w.out[w.starts_list[-1]:] == SENTINEL).all()


@pytest.mark.parametrize("kind,heads", [("tree", 64), ("latent", 64)])
def test_the_walk_sees_a_single_block(gpu, kind, heads):
    """The same with one block of a long context taken for another: the rows aimed there are wrong, and no others."""
    w = Walk(80, [(9000, 8)], heads, 1, 16, BF, kind)
    held = w.tables.clone()
    for step, block in ((0, 3), (7, 230), (11, 500)):
        tables = w.tables
        w.tables = held.clone()
        w.tables[0, block] = held[0, 5]
        aims, wrong = w.step(step)       # (compared with the other block's values where aimed at it)
        there = aims[0] // 16 == block
        assert bool(there.any()) == (step * 512 <= block * 16 < (step + 1) * 512)
        blk, off = held[0, aims[0] // 16].long(), aims[0] % 16
        want = w.pools[1][blk, 0, off] if kind == "tree" else w.pools[0][blk, off][..., :LATENT]
        off = differ(w.out[:8].view(8, heads, -1), want).any(-1)
        assert torch.equal(off, there)
        w.tables = tables


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("heads,seqs", [(3, [(1100, 1100)]), (2, [(300, 2300), (257, 257), (64, 900)]), (40, [(129, 400)] * 5),
                                        (1, [(2600, 2600)])])
def test_every_key_of_a_prompt(gpu, heads, seqs, dtype):
    p = Prompts(90 + heads, seqs, heads, dtype, extra=2, scale=1.0)
    g = torch.Generator(device="cuda").manual_seed(90)
    Tk = p.ks_list[-1]
    p.kv[:Tk, :, :D] = signs(g, Tk, heads, D).to(dtype)
    p.k_rope[:Tk] = signs(g, Tk, ROPE).to(dtype)
    keys = torch.cat([p.kv[:, :, :D], p.k_rope[:, None].expand(-1, heads, -1)], dim=-1)
    for s, (n, m) in enumerate(seqs):
        some = torch.randint(0, m, (64,), generator=g, device="cuda").unique()
        assert all(gap(keys[p.ks_list[s]:p.ks_list[s] + m, h], some) >= 40 for h in range(heads))
    total = torch.zeros((), dtype=torch.int64, device=gpu)
    seen = [torch.zeros(m, dtype=torch.bool, device=gpu) for _, m in seqs]
    head = torch.arange(heads, device=gpu)
    for step in range(48):
        aims = []
        for s, (n, m) in enumerate(seqs):
            a, b = p.qs_list[s], p.ks_list[s]
            i = torch.arange(n, device=gpu)[:, None]
            # itself and the keys right before it in turn, and all over what it attends
            at = (m - n + i - step // 2).expand(n, heads) if step % 2 else i * 61 + head * 17 + step * 53
            at = at % (m - n + i + 1)
            seen[s][at.flatten()] = True
            aims.append(at)
            p.q[a:a + n] = keys[b + at, head]
        p.out.fill_(SENTINEL)
        p.call()
        for s, at in enumerate(aims):
            a, b = p.qs_list[s], p.ks_list[s]
            total += differ(p.out[a:a + len(at)], p.kv[b + at, head, D:]).any(-1).sum()
    assert pkv.check_device_error() == 0
    assert int(total) == 0
    assert all(float(x.float().mean()) > 0.99 for x in seen)
