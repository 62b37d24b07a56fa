"""Host-side refusals of the calls on drafted tokens, latent caches and prompts: no GPU, nothing launched."""
import ctypes

import pytest

from paged_kv_cache_11_gb300 import _build, binding
from tests.test_abi import declared_functions

OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA = (binding.PKV_OK, binding.PKV_ERR_INVALID_ARG, binding.PKV_ERR_UNSUPPORTED,
                                             binding.PKV_ERR_WORKSPACE, binding.PKV_ERR_CUDA)
BIG = 1 << 62
Q, K, V, OUT, TAB, LEN, ST, MASK, WS = ((i + 1) << 40 for i in range(9))  # addresses that nothing reads


@pytest.fixture(scope="module")
def lib():
    _build.build_library()
    return binding._lib()


def test_entry_points_are_declared_and_exported(lib):
    names = {"paged_attention_tree", "paged_attention_tree_workspace_bytes", "paged_latent_append_rope",
             "paged_latent_decode", "paged_latent_decode_workspace_bytes", "latent_attention_prefill"}
    assert names <= set(declared_functions())
    import paged_kv_cache_11_gb300 as pkv
    assert all(hasattr(lib, n) and hasattr(pkv, n) for n in names)


def test_structs_have_the_headers_layout():
    assert ctypes.sizeof(binding.LatentDesc) == 24 and ctypes.sizeof(binding.LatentRopeDesc) == 64
    assert ctypes.sizeof(binding.PromptDesc) == 64 and binding.LatentRopeDesc.norm_eps.offset == 56
    assert binding.DEVERR_NAMES[10] == "query"


def _ref(d):
    return ctypes.byref(d) if d is not None else None


def _tree(lib, desc=0, q=Q, k=K, v=V, tab=TAB, width=8, lens=LEN, starts=ST, masks=MASK, seqs=4, tokens=9, heads=8, scale=0.1,
          out=OUT, ws=WS, ws_bytes=BIG):
    if desc == 0:
        desc = binding.CacheDesc(64, 2, 16, 128, binding.PKV_BF16)
    return lib.paged_attention_tree(q, k, v, tab, width, lens, starts, masks, seqs, tokens, heads, scale, out, _ref(desc), ws,
                                    ws_bytes, None)


def _latent(lib, desc=0, q=Q, c=K, tab=TAB, width=8, lens=LEN, starts=ST, masks=MASK, seqs=4, tokens=9, heads=8, scale=0.1,
            out=OUT, ws=WS, ws_bytes=BIG):
    if desc == 0:
        desc = binding.LatentDesc(64, 16, 512, 64, binding.PKV_BF16)
    return lib.paged_latent_decode(q, c, tab, width, lens, starts, masks, seqs, tokens, heads, scale, out, _ref(desc), ws,
                                   ws_bytes, None)


@pytest.mark.parametrize("call", [_tree, _latent])
def test_drafted_calls(lib, call):
    f = lambda **kw: call(lib, **kw)
    assert f(seqs=0, tokens=0) == OK and f(tokens=0) == OK
    assert f(seqs=0, tokens=9, starts=ST) == OK          # no sequence: no row is anyone's
    assert f(desc=None) == INVALID
    assert f(seqs=-1) == INVALID and f(seqs=65536) == INVALID and f(tokens=-1) == INVALID
    assert f(starts=None) == INVALID                     # 9 tokens of 4 sequences
    assert f(heads=0) == INVALID and f(heads=65536 * 2) == UNSUPPORTED
    assert f(width=0) == INVALID and f(width=1 << 30) == UNSUPPORTED
    assert f(tokens=1 << 30, heads=64) == UNSUPPORTED    # rows past 32 bits
    for s in (float("nan"), float("inf"), float("-inf")):
        assert f(scale=s) == INVALID
    for a in ("q", "tab", "lens", "out"):
        assert f(**{a: None}) == INVALID, a
    for a in ("q", "out"):
        assert f(**{a: Q + 8}) == INVALID, a
    assert f(tab=TAB + 2) == INVALID and f(lens=LEN + 2) == INVALID and f(starts=ST + 2) == INVALID
    assert f(masks=MASK + 4) == INVALID
    # from here on the device is asked for its size; without one the call ends there
    assert f(ws=None) in (WORKSPACE, CUDA) and f(ws_bytes=1000) in (WORKSPACE, CUDA) and f(ws=WS + 128) in (WORKSPACE, CUDA)


def test_tree_shapes(lib):
    d = lambda **kw: binding.CacheDesc(**(dict(num_blocks=64, num_kv_heads=2, block_size=16, head_dim=128, dtype=0) | kw))
    assert _tree(lib, desc=d(dtype=binding.PKV_E4M3)) == UNSUPPORTED and _tree(lib, desc=d(dtype=binding.PKV_FP32)) == UNSUPPORTED
    assert _tree(lib, desc=d(head_dim=64)) == UNSUPPORTED and _tree(lib, desc=d(block_size=8)) == UNSUPPORTED
    assert _tree(lib, desc=d(num_blocks=0)) == INVALID and _tree(lib, desc=d(num_kv_heads=3)) == INVALID
    assert _tree(lib, desc=d(num_blocks=1 << 40)) == UNSUPPORTED and _tree(lib, desc=d(num_blocks=1 << 27)) == UNSUPPORTED
    assert _tree(lib, k=None) == INVALID and _tree(lib, k=K + 4) == INVALID


def test_latent_shapes(lib):
    d = lambda **kw: binding.LatentDesc(**(dict(num_blocks=64, block_size=16, latent_dim=512, rope_dim=64, dtype=0) | kw))
    for kw in (dict(dtype=binding.PKV_FP32), dict(latent_dim=256), dict(rope_dim=32), dict(block_size=64),
               dict(num_blocks=1 << 31)):
        assert _latent(lib, desc=d(**kw)) == UNSUPPORTED, kw
    assert _latent(lib, desc=d(num_blocks=0)) == INVALID and _latent(lib, c=None) == INVALID and _latent(lib, c=K + 8) == INVALID


def test_workspaces_do_not_need_a_device_to_be_asked_for(lib):
    assert lib.paged_attention_tree_workspace_bytes() >= 0 and lib.paged_latent_decode_workspace_bytes() >= 0


def _append(lib, n=8, q=Q, kv=K, pos=TAB, table=LEN, norm=None, slots=ST, qo=OUT, kvo=None, cache=V, bs=16, dtype=0, cdesc=True,
            rdesc=True, **kw):
    c = binding.LatentDesc(64, bs, 512, 64, dtype)
    r = binding.LatentRopeDesc(**(dict(num_heads=4, interleaved=0, q_stride=256, q_head_stride=64, q_out_stride=256,
                                       q_out_head_stride=64, kv_stride=576, max_position=64, norm_eps=1e-6) | kw))
    return lib.paged_latent_append_rope(q, kv, pos, table, norm, slots, n, qo, kvo, cache, _ref(c) if cdesc else None,
                                        _ref(r) if rdesc else None, None)


def test_latent_append(lib):
    f = lambda **kw: _append(lib, **kw)
    assert f(n=0) == OK and f(n=0, bs=7) == OK
    assert f(n=-1) == INVALID and f(cdesc=False) == INVALID and f(rdesc=False) == INVALID
    assert f(dtype=binding.PKV_E4M3) == UNSUPPORTED
    for e in (-1.0, float("nan"), float("inf")):
        assert f(norm_eps=e) == INVALID
    for s in ("q_stride", "q_head_stride", "q_out_stride", "q_out_head_stride", "kv_stride"):
        assert f(**{s: 580}) == INVALID and f(**{s: -576}) == INVALID and f(**{s: 1 << 60}) == INVALID, s
    assert f(num_heads=-1) == INVALID and f(num_heads=70000) == UNSUPPORTED and f(n=1 << 40) == INVALID
    for a in ("q", "kv", "pos", "slots", "qo", "cache"):
        assert f(**{a: None}) == INVALID, a
    for a in ("q", "kv", "table", "qo", "cache", "norm", "kvo"):
        assert f(**{a: MASK + 8}) == INVALID, a
    assert f(pos=TAB + 4) == INVALID and f(slots=ST + 4) == INVALID and f(max_position=0) == INVALID
    # outputs over inputs: the same rows, or none of them
    assert f(qo=Q, q_out_stride=512) == INVALID and f(qo=Q + 64) == INVALID and f(qo=K) == INVALID
    assert f(kvo=K, kv_stride=1152) == INVALID and f(kvo=K + 576) == INVALID
    # heads or tokens of the output over one another
    assert f(q_out_head_stride=32) == INVALID and f(q_out_stride=0) == INVALID


def _prompt(lib, q=Q, kv=K, kr=V, qs=ST, ks=LEN, seqs=2, nq=100, nk=120, longest=60, scale=0.1, out=OUT, pdesc=True, **kw):
    d = binding.PromptDesc(**(dict(num_heads=4, dtype=0, nope_dim=128, rope_dim=64, value_dim=128, q_stride=768, q_head_stride=192,
                                   kv_stride=1024, kv_head_stride=256, k_rope_stride=576) | kw))
    return lib.latent_attention_prefill(q, kv, kr, qs, ks, seqs, nq, nk, longest, scale, out, _ref(d) if pdesc else None, None)


def test_prefill(lib):
    f = lambda **kw: _prompt(lib, **kw)
    assert f(seqs=0) == OK and f(nq=0, longest=0) == OK and f(longest=0) == OK
    assert f(pdesc=False) == INVALID and f(num_heads=0) == INVALID and f(num_heads=65536) == UNSUPPORTED
    for kw in (dict(dtype=2), dict(nope_dim=64), dict(rope_dim=32), dict(value_dim=64)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(seqs=-1), dict(seqs=65536), dict(nq=-1), dict(nk=-1), dict(longest=-1), dict(longest=101)):
        assert f(**kw) == INVALID, kw
    for s in (float("nan"), float("inf")):
        assert f(scale=s) == INVALID
    for s in ("q_stride", "q_head_stride", "kv_stride", "kv_head_stride", "k_rope_stride"):
        assert f(**{s: 772}) == INVALID and f(**{s: -8}) == INVALID and f(**{s: 1 << 50}) == INVALID, s
    for a in ("q", "kv", "kr", "qs", "ks", "out"):
        assert f(**{a: None}) == INVALID, a
    for a in ("q", "kv", "kr", "out"):
        assert f(**{a: MASK + 8}) == INVALID, a
    assert f(qs=ST + 2) == INVALID and f(ks=LEN + 2) == INVALID
    assert f(out=Q) == INVALID and f(out=Q + 1024) == INVALID
    assert f(nq=(1 << 31) - 1) == UNSUPPORTED


def test_the_binding_refuses_tensors_that_are_not_on_a_gpu(lib):
    import torch
    import paged_kv_cache_11_gb300 as pkv
    _build.build_marshal()
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    i32, i64 = (lambda *s: z(*s, dt=torch.int32)), (lambda *s: z(*s, dt=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attention_tree(z(3, 4, 128), z(2, 2, 16, 128), z(2, 2, 16, 128), i32(1, 2), i32(1), i32(2), None, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_latent_decode(z(1, 4, 576), z(2, 16, 576), i32(1, 2), i32(1), 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_latent_append_rope(z(1, 4, 64), z(1, 576), None, None, i64(1), z(2, 16, 576))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.latent_attention_prefill(z(3, 4, 192), z(3, 4, 256), z(3, 64), i32(2), i32(2), 0.1)
