"""Prompts whose tokens and heads lie in other orders, over one another or far apart: the same outputs as of contiguous ones, bit
by bit."""
import pytest
import torch

import paged_kv_cache_11_gb300 as pkv
from tests.test_latent_gpu import Prompts

pytestmark = pytest.mark.gpu

FORMS = {
    "heads first": lambda x: x.transpose(0, 1).contiguous().transpose(0, 1),
    "far apart": lambda x: torch.zeros(x.shape[0], x.shape[1] + 3, x.shape[2] + 24, dtype=x.dtype, device=x.device)
    .narrow(1, 2, x.shape[1]).narrow(2, 16, x.shape[2]).copy_(x),
    "one head for all": lambda x: x[:, :1].expand(-1, x.shape[1], -1),
    "one token for all": lambda x: x[:1].expand(x.shape[0], -1, -1),
}


@pytest.mark.parametrize("heads", [1, 5])
@pytest.mark.parametrize("form", list(FORMS))
def test_orders(gpu, form, heads):
    make = FORMS[form]
    for which in ("q", "kv", "k_rope"):
        p = Prompts(1, [(300, 300), (20, 150)], heads, torch.bfloat16)
        if which == "k_rope":
            if "head" in form:
                continue
            p.k_rope = make(p.k_rope[:, None])[:, 0]
        else:
            setattr(p, which, make(getattr(p, which)))
        got = p.call().clone()
        setattr(p, which, getattr(p, which).contiguous())
        want = p.call()
        assert pkv.check_device_error() == 0
        assert torch.equal(got, want), (form, which)
        p.check()
