"""Small weights beside large ones: what a cache of fp16 holds of them (drafted tokens, latent caches, prompts).

fp16 ends in steps of 2^-24, and a row's weights are held at seven binades above 2^0 for a score at its running maximum, which
the largest score reaches or passes: a weight is off by half a step of its own, 2^-11, or by 2^-25 / 2^7 = 2^-32 of the
largest.  So the bound of the helpers, which allows 2^-25 of the largest weight for each token, is tightened to 2^-32 here."""
import pytest
import torch

import paged_kv_cache_11_gb300 as pkv
from tests.drafted_helpers import D, Batch, attend64
from tests.test_latent_gpu import Prompts

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def tight(bound, n, v):
    """The helpers' bound of an fp16 output for n tokens of values v, with 2^-32 for their 2^-25."""
    return bound - (2.0 ** -25 - 2.0 ** -32) * n * v.abs().amax()


@pytest.mark.parametrize("kind,heads", [("tree", 8), ("tree", 300), ("latent", 16), ("latent", 128)])
@pytest.mark.parametrize("drop", [5, 10, 18, 20])
@pytest.mark.parametrize("seqs,L", [(1, 131072), (200, 8192)])
def test_a_sink_and_a_long_flat_tail(gpu, kind, heads, drop, seqs, L):
    """One token of value 0, and L - 1 of value 1 whose scores are `drop` below its own: contexts divided into many parts, and
    as many contexts as keep most of each in one part."""
    for at, dtype in ((0, FP), (L // 2 + 37, FP), (L - 1, FP), (0, BF)):
        b = Batch(40, [(L, 1)] * seqs, heads, 1, 32, dtype, kind, "chain", scale=1.0)
        b.q.zero_()
        b.q[..., 0] = 1.0
        blk, off = b.tables[:, at // 32].long(), at % 32
        for x in b.pools:
            x.fill_(1.0)
        if kind == "tree":
            b.pools[0].zero_()
            b.pools[0][blk, 0, off, 0] = drop
            b.pools[1][blk, 0, off] = 0.0
        else:
            b.pools[0][..., 0] = 0.0
            b.pools[0][blk, off] = 0.0
            b.pools[0][blk, off, 0] = drop
        out = b.call()
        assert pkv.check_device_error() == 0
        # every row and dim but the key's own is the same: one head in 64 bits
        one = torch.ones(1, 1, 1, dtype=torch.float64, device=gpu)
        key = torch.zeros(1, L, 1, dtype=torch.float64, device=gpu)
        key[0, at] = drop
        val = 1.0 - (torch.arange(L, device=gpu) == at).double()[None, :, None]
        y, bound = attend64(one, key, val, torch.ones(1, L, dtype=torch.bool, device=gpu), 1.0, dtype)
        y, bound = float(y), float(tight(bound, L, val) if dtype == FP else bound)
        got = out.double()[..., 1:] if kind == "latent" else out.double()
        assert float((got - y).abs().max()) <= bound, (dtype, y, float(got.min()), float(got.max()), bound)


def test_a_sink_and_a_long_flat_tail_in_a_prompt(gpu):
    m, n = 65536, 3
    for at in (0, 40000):
        for drop in (5, 17):
            p = Prompts(1, [(n, m)], 2, FP, scale=1.0)
            p.q.zero_(), p.kv.zero_(), p.k_rope.zero_()
            p.q[..., 0] = 1.0
            p.kv[at, :, 0] = drop
            p.kv[..., D:] = 1.0
            p.kv[at, :, D:] = 0.0
            out = p.call()
            assert pkv.check_device_error() == 0
            y, bound = p.expected(0)
            assert ((out.double() - y).abs() <= tight(bound, m, p.kv[..., D:].double())).all(), float(out.float().max())


@pytest.mark.parametrize("kind,heads,hkv", [("tree", 8, 2), ("tree", 64, 1), ("latent", 16, 1), ("latent", 128, 1)])
@pytest.mark.parametrize("scale", [0.02, 0.09, 0.6, 2.5])
def test_fp16_contexts(gpu, kind, heads, hkv, scale):
    """From nearly equal weights to a few that hold all of it; long and short contexts."""
    b = Batch(41, [(9000, 2), (700, 5), (40, 7), (129, 1)], heads, hkv, 16, FP, kind, "tree", scale=scale)
    b.call()
    assert pkv.check_device_error() == 0
    for s in range(4):
        y, bound = b.expected(s)
        got = b.out[b.starts_list[s]:b.starts_list[s] + b.counts[s]].double()
        assert ((got - y).abs() <= tight(bound, b.lens[s], b.rows(s)[1])).all(), s


def test_scores_that_climb(gpu):
    """Scores that climb by just less than what raises the running maximum: weights up to the top of fp16's range."""
    for kind in ("tree", "latent"):
        for step in (5.4, 5.6, 11.0):     # natural units; 8 in the exponent of 2 is 5.545
            L = 1200
            b = Batch(42, [(L, 3)], 16, 1, 16, FP, kind, "chain", scale=1.0)
            b.q.zero_()
            b.q[..., 0] = 1.0
            t = torch.arange(L, device=gpu)
            blk, off = b.tables[0, t // 16].long(), t % 16
            climb = (t // 128 * step).half()
            if kind == "tree":
                b.pools[0][blk, 0, off, 0] = climb
            else:
                b.pools[0][blk, off, 0] = climb
            b.call()
            assert pkv.check_device_error() == 0
            y, bound = b.expected(0)
            assert ((b.out[:3].double() - y).abs() <= tight(bound, L, b.rows(0)[1])).all(), (kind, step)
