"""The compiled binding of the rotating writes and the 8-bit cache: what it cannot pass on is an exception, not the end of
the process."""
import numpy as np
import pytest
import torch

import paged_kv_cache_11_gb300 as pkv
from tests.fp8_helpers import Case, decode_inputs, runs_of_tokens

pytestmark = pytest.mark.gpu


def test_a_table_too_wide_for_the_library(gpu):
    """No sequences, and rows of 2^31 block ids: the width does not fit the call's 32 bits."""
    d = {k: v.to(gpu) for k, v in decode_inputs(1, (40,), 4, 2, 16, torch.bfloat16).items()}
    d.update(q=d["q"][:0], context_lens=d["context_lens"][:0],
             block_tables=torch.empty((0, 2 ** 31), dtype=torch.int32, device=gpu))
    with pytest.raises(ValueError):
        pkv.paged_attention_decode_fp8(**d, scale=0.1, max_context_len=16)
    with pytest.raises(ValueError):
        pkv.paged_attention_decode_fp8(**d, scale=0.1)


def test_tensors_without_memory(gpu):
    """Inside vmap a tensor stands for many and has no address."""
    launches = pkv.launch_count()
    d = {k: v.to(gpu) for k, v in decode_inputs(2, (40, 20), 4, 2, 16, torch.bfloat16).items()}
    q = d.pop("q")
    with pytest.raises(RuntimeError):
        torch.func.vmap(lambda x: pkv.paged_attention_decode_fp8(x, **d, scale=0.1))(torch.stack([q, q]))
    slots, pos = runs_of_tokens(np.random.default_rng(1), [(0, 5)], 16, 4)
    for fp8 in (False, True):
        c = Case(3, 4, 2, 16, torch.bfloat16, 128, False, True, slots, pos, 4, fp8=fp8).to_dev(gpu)
        call = pkv.paged_kv_append_rope_fp8 if fp8 else pkv.paged_kv_append_rope
        k = c.pop("k")
        with pytest.raises(RuntimeError):
            torch.func.vmap(lambda x: call(k=x, **c))(torch.stack([k, k]))
    pairs = torch.tensor([[[0, 1]], [[1, 2]]], device=gpu)
    with pytest.raises(RuntimeError):
        torch.func.vmap(lambda x: pkv.copy_blocks_fp8(d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"], x))(pairs)
    assert pkv.launch_count() == launches
