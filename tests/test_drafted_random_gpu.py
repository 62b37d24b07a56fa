"""Random batches of the calls on drafted tokens, latent caches and prompts against their definitions in 64 bits, the calls
beside the package's others, and the refusals that need tensors of a GPU (PKV_SOAK=k: k times as many batches)."""
import os
import random

import pytest
import torch

import paged_kv_cache_11_gb300 as pkv
from tests.drafted_helpers import LATENT, ROW, Batch
from tests.test_latent_gpu import Prompts, Write

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
SOAK = int(os.environ.get("PKV_SOAK", "1"))


@pytest.mark.parametrize("seed", range(24 * SOAK))
@pytest.mark.parametrize("kind", ["tree", "latent"])
def test_random_batches(gpu, kind, seed):
    r = random.Random(1000 * seed + (kind == "tree"))
    if kind == "tree":
        heads, hkv = r.choice([(4, 1), (8, 8), (32, 8), (24, 3), (64, 8), (16, 1), (7, 7), (96, 1), (2, 2)])
    else:
        heads, hkv = r.choice([1, 3, 8, 16, 33, 40, 64, 65, 100, 128, 130]), 1
    most = r.choice([1, 2, 5, 16, 40, 64])
    top = int(2 ** r.uniform(0, 12 if heads < 64 else 10))
    seqs = []
    for _ in range(int(2 ** r.uniform(0, 5))):
        n = r.randint(0 if r.random() < 0.2 else 1, most)
        L = 0 if r.random() < 0.1 else max(n, r.randint(1, max(1, top)))
        seqs.append((L, n))
    b = Batch(seed, seqs, heads, hkv, r.choice([16, 32]), r.choice([BF, FP]), kind, r.choice(["tree", "chain", "random"]),
              extra=r.randint(1, 4), scale=r.choice([None, None, 0.3, -0.1]), width=r.choice([0, 0, 200]))
    b.call()
    assert pkv.check_device_error() == 0
    b.check()


@pytest.mark.parametrize("seed", range(16 * SOAK))
def test_random_prompts(gpu, seed):
    r = random.Random(seed)
    seqs = []
    for _ in range(r.randint(1, 6)):
        n = int(2 ** r.uniform(0, 10))
        seqs.append((n, max(0, n + r.choice([0, 0, 0, 1, 77, 500, -1, -n // 2]))))
    p = Prompts(seed, seqs, r.choice([1, 2, 5, 16]), r.choice([BF, FP]), extra=r.randint(0, 3), slices=r.random() < 0.5,
                scale=r.choice([None, 0.2, -0.1]), gap=r.choice([0, 5]))
    p.call()
    assert pkv.check_device_error() == 0
    p.check()


@pytest.mark.parametrize("seed", range(12 * SOAK))
def test_random_writes(gpu, seed):
    r = random.Random(seed)
    spans = [(r.randint(0, 300), int(2 ** r.uniform(0, 6))) for _ in range(r.randint(1, 5))]
    total = sum(n for _, n in spans)
    w = Write(seed, spans, r.choice([0, 1, 4, 16, 31, 128]), r.choice([1, 16, 32]), r.choice([BF, FP]), r.random() < 0.5,
              r.random() < 0.7, r.random() < 0.8, pads=sorted(r.sample(range(total), min(total, r.randint(0, 3)))))
    kv_out = torch.zeros(w.n, ROW, dtype=w.dtype, device=gpu)
    q = w.call(kv_out=kv_out)
    assert pkv.check_device_error() == 0
    w.check(q, kv_out)


def test_as_decode_attention(gpu):
    """One token a sequence: what paged_attention_decode gives, to the output's rounding and that of the weights."""
    b = Batch(3, [(1, 1), (700, 1), (33, 1), (0, 1)], 32, 8, 16, BF, "tree", "chain", starts=False)
    out = b.call(out=None)
    want = pkv.paged_attention_decode(b.q, *b.pools, b.tables, b.context_lens, b.scale)
    v = torch.nan_to_num(b.pools[1].float()).abs().max()
    assert (out.float() - want).abs().max() <= 2 * 2.0 ** -8 * v     # u (A + |y|) + u |y| and some, A <= max |v|
    assert pkv.check_device_error() == 0


def test_more_than_the_average_of_a_batch(gpu):
    """The rows of a sequence go by the batch's average, whichever way: one long tree among single tokens, and the reverse."""
    for seqs in ([(500, 64)] + [(300, 1)] * 40, [(500, 1)] + [(200, 9)] * 6):
        for heads in (16, 40):
            b = Batch(5, seqs, heads, 1, 16, BF, "latent", "tree", extra=2)
            b.call()
            assert pkv.check_device_error() == 0
            b.check(only=[0, 1, len(seqs) - 1])


def test_refusals_of_tensors(gpu):
    b = Batch(1, [(40, 3), (20, 2)], 8, 2, 16, BF, "tree", "tree")
    good = dict(q=b.q, k_cache=b.pools[0], v_cache=b.pools[1], block_tables=b.tables, context_lens=b.context_lens,
                query_starts=b.starts, tree_masks=b.masks, scale=b.scale)
    ok = pkv.paged_attention_tree(**good)
    for bad in (dict(q=b.q.half()), dict(q=b.q[..., :64]), dict(q=b.q.transpose(0, 1)), dict(v_cache=b.pools[1][:-1]),
                dict(block_tables=b.tables.long()), dict(block_tables=b.tables[:, ::2]), dict(context_lens=b.context_lens[:1]),
                dict(query_starts=b.starts.long()), dict(query_starts=b.starts[:2]), dict(query_starts=None),
                dict(tree_masks=b.masks.int()), dict(tree_masks=b.masks[:3]), dict(tree_masks=b.masks.cpu()), dict(scale="x"),
                dict(out=torch.empty_like(ok).half()), dict(out=ok[:2])):
        with pytest.raises((ValueError, TypeError)):
            pkv.paged_attention_tree(**(good | bad))
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_attention_tree(**good, workspace=torch.empty(256, dtype=torch.uint8, device=gpu))
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_attention_tree(**good, out=b.q)
    c = Batch(2, [(40, 3), (20, 2)], 8, 1, 16, BF, "latent", "tree")
    good = dict(q=c.q, cache=c.pools[0], block_tables=c.tables, context_lens=c.context_lens, scale=c.scale, query_starts=c.starts)
    for bad in (dict(q=c.q[..., :LATENT].contiguous()), dict(cache=c.pools[0][..., :LATENT].contiguous()),
                dict(cache=c.pools[0].half()), dict(query_starts=None), dict(out=torch.empty_like(c.q))):
        with pytest.raises(ValueError):
            pkv.paged_latent_decode(**(good | bad))
    w = Write(3, [(0, 5)], 4, 16, BF)
    pos, slots = w.pos.cuda(), w.slots.cuda()
    good = dict(q=w.q, kv=w.kv, positions=pos, cos_sin=w.table, slot_mapping=slots, cache=w.cache, kv_norm=w.norm)
    for bad in (dict(q=w.q[:3]), dict(kv=w.kv[:, 8:]), dict(kv=w.kv.float()), dict(positions=None), dict(positions=pos.int()),
                dict(cos_sin=w.table[:, :32].contiguous()), dict(slot_mapping=slots.int()), dict(kv_norm=w.norm.float()),
                dict(kv_out=torch.empty(5, LATENT, dtype=BF, device=gpu)), dict(q_out=w.q.float()), dict(q=None, q_out=w.q)):
        with pytest.raises(ValueError):
            pkv.paged_latent_append_rope(**(good | bad))
    p = Prompts(4, [(9, 9)], 2, BF)
    good = dict(q=p.q, kv=p.kv, k_rope=p.k_rope, query_starts=p.qs, key_starts=p.ks, scale=0.1)
    for bad in (dict(kv=p.kv[:, :1]), dict(k_rope=p.k_rope[:5]), dict(kv=p.kv.half()), dict(key_starts=p.ks[:1]),
                dict(query_starts=p.qs.long()), dict(out=torch.empty(9, 2, 64, dtype=BF, device=gpu))):
        with pytest.raises(ValueError):
            pkv.latent_attention_prefill(**(good | bad))
    with pytest.raises(pkv.PagedKVError):
        pkv.latent_attention_prefill(**good, max_query_len=10)
    assert pkv.check_device_error() == 0
