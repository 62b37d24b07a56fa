"""Batches of many prompts: where each one's strips of 256 queries lie among those of all, whatever bound of the longest is
given."""
import pytest
import torch

import paged_kv_cache_11_gb300 as pkv
from tests.drafted_helpers import SENTINEL
from tests.test_latent_gpu import Prompts, run

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def batch(seed, count, longest):
    """Prompts of 0 to `longest` tokens, some behind a prefix, some with fewer keys than queries, a long one among them."""
    g = torch.Generator().manual_seed(seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    seqs = []
    for _ in range(count):
        n = r(0, longest) if r(0, 3) else 0
        seqs.append((n, max(0, n + (r(0, 40) if r(0, 1) else -r(0, 3)))))
    seqs[r(0, count - 1)] = (700, 730)
    return seqs


@pytest.mark.parametrize("count,longest,heads", [(2, 600, 3), (31, 300, 2), (32, 9, 40), (33, 300, 2), (64, 20, 9), (65, 20, 9),
                                                 (128, 300, 1), (511, 40, 3), (512, 40, 3), (513, 40, 3), (1100, 20, 5),
                                                 (3000, 5, 2)])
def test_batches_of_many_prompts(gpu, count, longest, heads):
    seqs = batch(count, count, longest)
    p = Prompts(count, seqs, heads, BF, extra=3, gap=2)
    run(p)
    big = [i for i, (n, _) in enumerate(seqs) if n == 700]
    some = sorted(set(range(0, count, max(1, count // 60))) | set(big) | {count - 1})
    p.check(only=some)
    first = p.out.clone()
    p.out.fill_(SENTINEL)
    run(p, max_query_len=None)
    assert torch.equal(p.out, first)
    used = p.out[p.qs_list[0]:p.qs_list[-1]]
    assert not (used == SENTINEL).flatten(1).all(1).any()      # every query's row was written


def test_the_most_prompts_of_a_call(gpu):
    count = 65535
    seqs = [(i % 3 > 0, 1 + i % 2) for i in range(count)]
    seqs = [(int(n), m) for n, m in seqs]
    seqs[65000] = (300, 310)
    p = Prompts(1, seqs, 2, BF, extra=1)
    run(p, max_query_len=None)
    p.check(only=list(range(0, count, 2111)) + [64999, 65000, 65001, 65533, 65534])
    assert not (p.out[:p.qs_list[-1]] == SENTINEL).flatten(1).all(1).any()


@pytest.mark.parametrize("count", [40, 600])
def test_bad_metadata_among_many(gpu, count):
    seqs = [(5 + i % 7, 9 + i % 7) for i in range(count)]
    seqs[3], seqs[20] = (300, 300), (600, 610)
    make = lambda: Prompts(2, seqs, 3, BF, extra=2)
    p = make()
    run(p, expect=10, max_query_len=299)
    p.check(only=list(range(0, count, count // 20)) + [2, 3, 4, 19, 20, 21, count - 1], zeros=[3, 20])
    p = make()
    p.ks[count // 2] = -5
    run(p, expect=10)
    p.check(only=[0, 3, 20, count // 2 - 1, count // 2, count // 2 + 1, count - 1], zeros=[count // 2 - 1, count // 2])
    p = make()
    p.qs[30] = 1 << 30
    run(p, expect=10)
    p.check(only=[0, 3, 20, 28, 31, 32, count - 1])
    assert (p.out[p.qs_list[29]:p.qs_list[31]] == SENTINEL).all()
    p = make()
    p.qs[:] = torch.where(torch.arange(count + 1, device=gpu) % 2 == 0, 0, p.qs[-1])     # every other prompt is all of them
    out = p.call(max_query_len=None)
    torch.cuda.synchronize()
    assert pkv.check_device_error() == 10 and out.shape == p.q.shape[:2] + (128,)


def test_the_time_without_a_bound_of_the_longest(gpu):
    """1024 prompts of 64 tokens with 8 heads: 8192 strips, where a place for each prompt and each strip that one prompt of all
    the tokens would have is 2 million."""
    p = Prompts(3, [(64, 64)] * 1024, 8, BF)
    times = {}
    for bound in (64, None):
        t = []
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            p.call(max_query_len=bound)
            b.record()
            b.synchronize()
            t.append(a.elapsed_time(b))
        times[bound] = min(t[1:])
    assert pkv.check_device_error() == 0
    p.check(only=[0, 511, 1023])
    assert times[None] <= 2 * times[64], times


def test_the_time_of_a_batch_most_of_which_is_empty(gpu):
    """20000 sequences, 50 of which have new tokens, against those 50 alone.  The lengths of all are read (20 us at most), and the
    strips that the tokens could make, one each, are looked through: 64 heads of them, less the 50, over the SMs, each a claim
    of 2 us at most.  (A place for each sequence would be 20000 for a head.)"""
    some = [(3 + i % 9, 40) for i in range(50)]
    times = []
    for seqs in (some, [some[i // 400] if i % 400 == 7 else (0, 0) for i in range(20000)]):
        p = Prompts(5, seqs, 64, BF)
        t = []
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            pkv.latent_attention_prefill(p.q, p.kv, p.k_rope, p.qs, p.ks, p.scale, out=p.out)
            b.record()
            b.synchronize()
            t.append(a.elapsed_time(b))
        times.append(min(t[1:]))
        assert pkv.check_device_error() == 0
        p.check(only=range(7, len(seqs), 400) if len(seqs) > 50 else None)
    claims = (p.q.shape[0] - 50) * 64 / torch.cuda.get_device_properties(gpu).multi_processor_count
    assert times[1] <= times[0] + 0.02 + 0.002 * claims, (times, claims)
