"""Host-side refusals of the rotating cache writes and the e4m3 cache calls: no GPU, nothing launched."""
import ctypes

import pytest

from paged_kv_cache_11_gb300 import _build, binding
from tests.test_abi import declared_functions

OK, INVALID, UNSUPPORTED, WORKSPACE = (binding.PKV_OK, binding.PKV_ERR_INVALID_ARG, binding.PKV_ERR_UNSUPPORTED,
                                       binding.PKV_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    _build.build_library()
    return binding._lib()


def test_entry_points_are_declared_and_exported(lib):
    names = {"paged_kv_append_rope", "paged_kv_append_rope_fp8", "paged_attention_decode_fp8", "copy_blocks_fp8"}
    assert names <= set(declared_functions())
    import paged_kv_cache_11_gb300 as pkv
    assert all(hasattr(lib, n) and hasattr(pkv, n) for n in names)


def _desc(dtype=binding.PKV_E4M3, **kw):
    d = dict(num_blocks=64, num_kv_heads=2, block_size=16, head_dim=128, dtype=dtype)
    d.update(kw)
    return binding.CacheDesc(**d)


def _rope(**kw):
    d = dict(num_q_heads=4, dtype=binding.PKV_BF16, q_stride=512, k_stride=256, v_stride=256, max_position=64, rot_dim=128,
             interleaved=0, norm_eps=1e-6)
    d.update(kw)
    return binding.RopeDesc(**d)


Q, K, V, QOUT = 1 << 30, 2 << 30, 3 << 30, 4 << 30  # addresses that nothing reads


def _append(lib, fp8, desc, rope, n=8, q=Q, k=K, v=V, pos=16, table=16, qn=None, kn=None, slots=16, qout=QOUT, kc=16,
            vc=16, ks=16, vs=16):
    pools = (kc, vc, ks, vs) if fp8 else (kc, vc)
    f = lib.paged_kv_append_rope_fp8 if fp8 else lib.paged_kv_append_rope
    return f(q, k, v, pos, table, qn, kn, slots, n, qout, *pools, ctypes.byref(desc) if desc else None,
             ctypes.byref(rope) if rope else None, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_rope_host_validation(lib, fp8):
    good = binding.PKV_E4M3 if fp8 else binding.PKV_BF16
    d, r = _desc(good), _rope()
    call = lambda desc=d, rope=r, **kw: _append(lib, fp8, desc, rope, **kw)
    assert call(n=0) == OK
    assert call(n=-1) == INVALID
    assert _append(lib, fp8, None, r) == INVALID and _append(lib, fp8, d, None) == INVALID
    assert call(desc=_desc(binding.PKV_BF16 if fp8 else binding.PKV_E4M3)) == UNSUPPORTED
    assert call(desc=_desc(good, head_dim=64)) == UNSUPPORTED
    assert call(desc=_desc(good, num_kv_heads=0)) == INVALID
    assert call(desc=_desc(good, num_blocks=1 << 60)) == INVALID            # byte offsets past 64 bits
    assert call(rope=_rope(dtype=binding.PKV_FP32)) == UNSUPPORTED
    assert call(rope=_rope(rot_dim=136)) == UNSUPPORTED
    assert call(rope=_rope(rot_dim=24)) == UNSUPPORTED
    assert call(rope=_rope(rot_dim=-16)) == INVALID
    assert call(rope=_rope(norm_eps=-1.0)) == INVALID
    assert call(rope=_rope(norm_eps=float("nan"))) == INVALID
    assert call(rope=_rope(norm_eps=float("inf"))) == INVALID
    assert call(rope=_rope(num_q_heads=-1)) == INVALID
    assert call(rope=_rope(max_position=0)) == INVALID
    for s in ("q_stride", "k_stride", "v_stride"):
        assert call(rope=_rope(**{s: 260})) == INVALID                      # rows off the 16-byte grid
        assert call(rope=_rope(**{s: -512})) == INVALID
        assert call(rope=_rope(**{s: 1 << 60})) == INVALID
    for a in ("q", "k", "v", "pos", "table", "slots", "qout", "kc", "vc") + (("ks", "vs") if fp8 else ()):
        assert call(**{a: None}) == INVALID, a
    for a in ("q", "k", "v", "table", "kc", "vc", "qn", "kn"):
        assert call(**{a: Q + 8}) == INVALID, a
    assert call(pos=20) == INVALID and call(slots=20) == INVALID
    assert call(n=1 << 40) == INVALID
    # q_out over q's rows, but not row by row; over k's or v's
    assert call(rope=_rope(q_stride=1024), qout=Q) == INVALID
    assert call(qout=Q + 1024) == INVALID
    assert call(qout=K - 1024) == INVALID and call(qout=V + 2048) == INVALID
    if fp8:
        assert call(desc=_desc(block_size=8)) == UNSUPPORTED
        assert call(ks=18) == INVALID
    else:
        assert call(rope=_rope(dtype=binding.PKV_FP16)) == INVALID          # not the cache's type


def _decode(lib, desc, num_seqs=1, hq=4, max_ctx=16, out_dtype=binding.PKV_FP32, P=0, ws=None, ws_bytes=0, maxb=4,
            qd=binding.PKV_BF16, scale=0.1, **kw):
    a = dict(q=16, k=16, v=16, ks=16, vs=16, bt=16, cl=16, out=16)
    a.update(kw)
    return lib.paged_attention_decode_fp8(a["q"], qd, a["k"], a["v"], a["ks"], a["vs"], a["bt"], maxb, a["cl"], num_seqs,
                                          hq, max_ctx, scale, a["out"], out_dtype, ctypes.byref(desc) if desc else None,
                                          P, ws, ws_bytes, None)


def test_decode_fp8_host_validation(lib):
    d = _desc()
    assert _decode(lib, d, num_seqs=0) == OK
    assert _decode(lib, None) == INVALID
    assert _decode(lib, _desc(binding.PKV_BF16)) == UNSUPPORTED
    assert _decode(lib, _desc(head_dim=64)) == UNSUPPORTED
    assert _decode(lib, _desc(block_size=8)) == UNSUPPORTED
    assert _decode(lib, _desc(num_blocks=1 << 60)) == INVALID
    assert _decode(lib, d, qd=binding.PKV_FP32) == UNSUPPORTED
    assert _decode(lib, d, qd=binding.PKV_E4M3) == UNSUPPORTED
    assert _decode(lib, d, out_dtype=binding.PKV_E4M3) == INVALID
    assert _decode(lib, d, hq=3) == INVALID
    assert _decode(lib, d, num_seqs=65536) == INVALID
    assert _decode(lib, d, max_ctx=65) == INVALID
    assert _decode(lib, d, max_ctx=-1) == INVALID
    assert _decode(lib, d, P=24) == INVALID and _decode(lib, d, P=-16) == INVALID
    assert _decode(lib, d, scale=float("nan")) == INVALID and _decode(lib, d, scale=float("inf")) == INVALID
    for a in ("q", "k", "v", "ks", "vs", "bt", "cl", "out"):
        assert _decode(lib, d, **{a: None}) == INVALID, a
        assert _decode(lib, d, **{a: 18}) == INVALID, a
    assert _decode(lib, d, max_ctx=64, P=16) == WORKSPACE
    assert _decode(lib, d, max_ctx=64, P=16, ws=256, ws_bytes=64) == WORKSPACE
    assert _decode(lib, d, max_ctx=64, P=16, ws=264, ws_bytes=1 << 30) == WORKSPACE


def test_copy_blocks_fp8_host_validation(lib):
    d = _desc()
    arr, bad = (ctypes.c_void_p * 1)(16), (ctypes.c_void_p * 1)(20)
    odd, null = (ctypes.c_void_p * 1)(18), (ctypes.c_void_p * 1)(None)
    f = lambda k=arr, v=arr, ks=arr, vs=arr, layers=1, pairs=16, n=3, desc=d: lib.copy_blocks_fp8(
        k, v, ks, vs, layers, pairs, n, ctypes.byref(desc) if desc else None, None)
    assert f(n=0) == OK and f(layers=0) == OK
    assert f(layers=-1) == INVALID and f(n=-1) == INVALID and f(desc=None) == INVALID
    assert f(desc=_desc(binding.PKV_FP16)) == UNSUPPORTED
    assert f(pairs=None) == INVALID and f(pairs=20) == INVALID
    for a in ("k", "v"):
        assert f(**{a: bad}) == INVALID and f(**{a: null}) == INVALID and f(**{a: None}) == INVALID
    for a in ("ks", "vs"):
        assert f(**{a: odd}) == INVALID and f(**{a: null}) == INVALID and f(**{a: None}) == INVALID


def test_other_calls_refuse_an_e4m3_pool(lib):
    d = _desc()
    assert lib.paged_kv_append(16, 16, 16, 4, 16, 16, ctypes.byref(d), None) == UNSUPPORTED
    arr = (ctypes.c_void_p * 1)(16)
    assert lib.copy_blocks(arr, arr, 1, 16, 3, ctypes.byref(d), None) == UNSUPPORTED
    assert lib.compact_tokens(16, 16, 4, 16, 16, ctypes.byref(d), None) == UNSUPPORTED


def test_binding_refuses_cpu_tensors():
    import torch
    import paged_kv_cache_11_gb300 as pkv
    c8 = torch.zeros(4, 1, 16, 128, dtype=torch.float8_e4m3fn)
    s = torch.ones(4, 1)
    x = torch.zeros(2, 1, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        pkv.paged_kv_append_rope_fp8(x, x, x, None, None, i, c8, c8, s, s)
    with pytest.raises(ValueError):
        pkv.paged_attention_decode_fp8(x, c8, c8, s, s, i.int()[:, None], i.int(), 0.1)
    with pytest.raises(ValueError):
        pkv.copy_blocks_fp8(c8, c8, s, s, i[None])
