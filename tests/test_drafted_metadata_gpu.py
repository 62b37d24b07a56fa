"""Bad metadata of drafted tokens beside sequences that are in order."""
import pytest
import torch

import paged_kv_cache_11_gb300 as pkv
from tests.drafted_helpers import SENTINEL, Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,heads,hkv", [("tree", 128, 2), ("tree", 40, 40), ("latent", 64, 1)])
@pytest.mark.parametrize("L", [512, 300, 64])
@pytest.mark.parametrize("seqs", [6, 16, 40])
def test_sequences_over_one_another(gpu, kind, heads, hkv, L, seqs):
    """query_starts 0, 64, 0, 64, ...: every other sequence's are out of order, and those between name the same rows, more
    units than the rows alone would make.  Where all of them read one context, its outputs come out, whoever writes them."""
    b = Batch(50, [(L, 64)], heads, hkv, 16, torch.bfloat16, kind, "tree", extra=2)
    starts = torch.tensor([0, 64] * ((seqs + 2) // 2), dtype=torch.int32, device=gpu)[:seqs + 1]
    tables, lens = b.tables.expand(seqs, -1).contiguous(), b.context_lens.expand(seqs).contiguous()
    for _ in range(2):
        b.out.fill_(SENTINEL)
        if kind == "tree":
            pkv.paged_attention_tree(b.q, *b.pools, tables, lens, starts, b.masks, b.scale, out=b.out)
        else:
            pkv.paged_latent_decode(b.q, *b.pools, tables, lens, b.scale, query_starts=starts, tree_masks=b.masks, out=b.out)
        assert pkv.check_device_error() == 10
        b.check()
