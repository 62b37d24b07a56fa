"""Block operations on latent pools: seen as one KV head of 576 values, [num_blocks, 1, block_size, 576], two layers' pools stand
where a layer's K and V do (or one pool for both)."""
import pytest
import torch

import paged_kv_cache_11_gb300 as pkv
from tests.drafted_helpers import ROW, Batch

pytestmark = pytest.mark.gpu


def view(pool):
    return pool.view(pool.shape[0], 1, pool.shape[1], ROW)


def pairs_of(pools):
    """The layers as (K, V) arguments: in twos, an odd last one for both."""
    return [view(p) for p in pools[0::2]], [view(p) for p in pools[1::2]] + ([view(pools[-1])] if len(pools) % 2 else [])


@pytest.mark.parametrize("layers", [1, 2, 3])
@pytest.mark.parametrize("bs,dtype", [(16, torch.bfloat16), (32, torch.float16)])
def test_copy_and_swap(gpu, layers, bs, dtype):
    g = torch.Generator(device=gpu).manual_seed(layers)
    pools = [torch.randn(40, bs, ROW, generator=g, device=gpu).to(dtype) for _ in range(layers)]
    expect = [p.clone() for p in pools]
    ids = torch.tensor([[3, 20], [3, 21], [0, 39], [17, 5]], device=gpu)
    pkv.copy_blocks(*pairs_of(pools), ids)
    for e in expect:
        e[ids[:, 1]] = e[ids[:, 0]]
    assert pkv.check_device_error() == 0
    assert all(torch.equal(p, e) for p, e in zip(pools, expect))
    host = [torch.zeros(8, bs, ROW, dtype=dtype).pin_memory() for _ in range(layers)]
    out = torch.tensor([[20, 1], [39, 7], [2, 0]], device=gpu)
    pkv.swap_blocks(*pairs_of(pools), *pairs_of(host), out)
    torch.cuda.synchronize()
    assert pkv.check_device_error() == 0
    for h, e in zip(host, expect):
        assert torch.equal(h[out[:, 1].cpu()], e[out[:, 0]].cpu()) and (h[[2, 3, 4, 5, 6]] == 0).all()
    pkv.swap_blocks(*pairs_of(host), *pairs_of(pools), torch.tensor([[1, 30], [7, 31]], device=gpu))
    assert pkv.check_device_error() == 0
    for p, e in zip(pools, expect):
        assert torch.equal(p[30], e[20]) and torch.equal(p[31], e[39])


@pytest.mark.parametrize("both", [True, False])
def test_compaction(gpu, both):
    a, b = (torch.randn(12, 16, ROW, device=gpu).bfloat16() for _ in range(2))
    b = a if both else b
    ea, eb = a.clone(), b.clone()
    src = torch.tensor([5, 17, 33, 80, -1, 100], device=gpu)
    dst = torch.tensor([160, 161, 162, 175, 3, -1], device=gpu)
    pkv.compact_tokens(src, dst, view(a), view(b))
    assert pkv.check_device_error() == 0
    for p, e in ((a, ea), (b, eb)):
        e.view(-1, ROW)[dst[:4]] = e.view(-1, ROW)[src[:4]]
        assert torch.equal(p, e)


def test_a_fork_attends_what_was_copied(gpu):
    """A sequence forked with its last block copied: the same outputs from the copy."""
    b = Batch(95, [(300, 3)], 16, 1, 16, torch.bfloat16, "latent", "tree", spare=3)
    first = b.call(out=None)
    used = set(b.tables[0, :19].tolist())
    free = next(i for i in range(b.pools[0].shape[0]) if i not in used)
    pkv.copy_blocks(*pairs_of(b.pools), torch.tensor([[int(b.tables[0, 18]), free]], device=gpu))
    b.tables[0, 18] = free
    assert torch.equal(b.call(out=None), first)
    assert pkv.check_device_error() == 0
