"""The most sequences that the calls on drafted tokens take."""
import pytest
import torch

import paged_kv_cache_11_gb300 as pkv
from tests.drafted_helpers import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,heads,hkv", [("tree", 2, 1), ("latent", 3, 1)])
def test_the_most_sequences_of_a_call(gpu, kind, heads, hkv):
    """65535, some of them empty or without drafted tokens, a long one and a tree of 64 among them."""
    count = 65535
    seqs = [(3 + i % 15, 1 + i % 3) if i % 7 else ((0, 1) if i % 2 else (9, 0)) for i in range(count)]
    seqs[40000], seqs[65534] = (5000, 2), (130, 64)
    b = Batch(70, seqs, heads, hkv, 16, torch.bfloat16, kind, "tree", extra=1)
    b.call()
    assert pkv.check_device_error() == 0
    b.check(only=list(range(0, count, 1777)) + [1, 7, 39999, 40000, 40001, 65533, 65534])
    empty = torch.tensor([b.starts_list[s] for s in range(count) if b.lens[s] == 0], device=gpu)
    assert (b.out[empty] == 0).all()
    b.lens[33333], b.context_lens[33333] = -1, -1       # an error among them is found
    b.call()
    assert pkv.check_device_error() == 3
    b.check(only=[33332, 33334, 40000], zeros=[])
    a = b.starts_list[33333]
    assert (b.out[a:a + b.counts[33333]] == 0).all()
