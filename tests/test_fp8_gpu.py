"""Decode attention over e4m3 pools and their copy-on-write copies, against their definitions in 64 bits."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_11_gb300 as pkv
from tests.fp8_helpers import D, Case, cos_sin_table, decode_inputs, decode_ref, runs_of_tokens, to64

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
SCALE = D ** -0.5


def _dev(inp, gpu):
    return {k: v.to(gpu) for k, v in inp.items()}


def _check(inp, gpu, out_dtype=F32, scale=SCALE, heads=None, **kw):
    out = pkv.paged_attention_decode_fp8(**_dev(inp, gpu), scale=scale, out_dtype=out_dtype, **kw)
    assert pkv.check_device_error() == 0
    ref, tol = decode_ref(inp, scale, out_dtype, heads)
    got = to64(out)
    sel = slice(None) if heads is None else list(heads)
    err = np.abs(got - ref)[:, sel]
    assert (err <= tol[:, sel]).all(), (err - tol[:, sel]).max()
    return out


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lens", [(1,), (0, 1, 15, 16, 17), (31, 32, 33, 0, 63, 64, 65), (129, 700, 5)])
def test_lengths(gpu, lens, dtype, bs):
    _check(decode_inputs(len(lens) + bs, lens, 4, 1, bs, dtype), gpu)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (12, 2), (24, 3), (16, 1), (32, 1), (40, 2), (9, 1)])
@pytest.mark.parametrize("bs", [16, 32])
def test_head_groups(gpu, hq, hkv, bs):
    _check(decode_inputs(hq + bs, (40, 333, 0, 6), hq, hkv, bs, BF), gpu)


@pytest.mark.parametrize("P", [0, 16, 32, 64, 512, 4096])
def test_partitions(gpu, P):
    inp = decode_inputs(P, (1500, 0, 700, 33, 1), 8, 2, 16, BF)
    _check(inp, gpu, partition_size=P)


@pytest.mark.parametrize("P", [640, 768, 896, 1280, 1536, 2048])
def test_partitions_that_the_automatic_choice_takes(gpu, P):
    _check(decode_inputs(P, (P - 1, P, P + 1, 2 * P + 17, 0, 1), 4, 1, 16, BF), gpu, partition_size=P)
    _check(decode_inputs(P + 1, (3 * P + 33, 5), 2, 2, 32, FP), gpu, partition_size=P)


@pytest.mark.parametrize("n,longest,hq,hkv,bs", [(1, 9000, 8, 1, 16), (40, 700, 4, 2, 32), (9, 3000, 16, 1, 16), (3, 6000, 3, 3, 32)])
def test_automatic_partitions_of_ragged_batches(gpu, n, longest, hq, hkv, bs):
    lens = np.random.default_rng(n).integers(0, longest + 1, n).tolist()
    lens[0] = longest
    _check(decode_inputs(n + 60, lens, hq, hkv, bs, BF), gpu)


@pytest.mark.parametrize("out_dtype", [F32, BF, FP])
@pytest.mark.parametrize("P", [0, 64])
def test_output_types(gpu, out_dtype, P):
    _check(decode_inputs(3, (600, 50, 0), 6, 2, 32, FP), gpu, out_dtype=out_dtype, partition_size=P)


@pytest.mark.parametrize("bs", [16, 32])
def test_scales_far_apart(gpu, bs):
    """Block scales that are no powers of two and spread over many orders: each block counts by its own."""
    _check(decode_inputs(17, (500, 90, 1), 8, 2, bs, BF, wild_scales=True), gpu)


@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("vs", [(0.0, 2.0 ** -64, 1.0, 2.0 ** -30, -1.0, 0.0, 2.0 ** 20), (0.0,), (0.3, 0.29, 0.31, 5.0),
                                (2.0 ** -64, 2.0 ** -63, 0.0), (-0.5, 0.5, -0.25, 1.0)])
def test_scales_of_any_sign_and_size(gpu, vs, order):
    inp = decode_inputs(23, (700, 90, 16), 8, 2, 16, BF)
    n = inp["v_scales"].shape[0]
    scales = torch.tensor((vs * n)[:n])
    inp["v_scales"][:] = (scales if order > 0 else scales.flip(0))[:, None]
    inp["k_scales"][::3] = 0
    _check(inp, gpu)
    _check(inp, gpu, partition_size=64)


@pytest.mark.parametrize("at", [0, 3, 20])
def test_a_block_of_huge_values_without_weight(gpu, at):
    """Values 2^40 times the others' that no weight reaches: the output keeps the others' full precision."""
    inp = decode_inputs(24, (500,), 4, 1, 16, BF)
    b = int(inp["block_tables"][0, at])
    inp["q"][:] = inp["q"][:, :1].abs()
    inp["k_cache"].view(torch.uint8)[b] |= 0x80                       # every key of the block against the query
    inp["k_scales"][b] = 2.0
    inp["v_scales"][b] = 2.0 ** 40
    _check(inp, gpu)


@pytest.mark.parametrize("out_dtype", [F32, BF])
@pytest.mark.parametrize("hq,bs", [(4, 16), (4, 32), (16, 16)])
@pytest.mark.parametrize("at", [0, 3, 14])
@pytest.mark.parametrize("kind", ["no weight", "zeros"])
@pytest.mark.parametrize("e", [62, 64])
def test_a_block_of_far_larger_scale_that_adds_nothing(gpu, e, kind, at, hq, bs, out_dtype):
    """A block whose scale is 2^62 or 2^64 times the others', without weight or of zeros: the others keep all they add,
    whether it comes before them or after."""
    inp = decode_inputs(61, (500,), hq, 1, bs, BF)
    b = int(inp["block_tables"][0, at])
    inp["v_scales"][:] = 1.0
    inp["v_scales"][b] = 2.0 ** e
    if kind == "zeros":
        inp["v_cache"].view(torch.uint8)[b] = 0
    else:
        inp["q"][:] = inp["q"][:, :1].abs()
        inp["k_cache"].view(torch.uint8)[b] |= 0x80                   # every key of the block against the query
        inp["k_scales"][b] = 2.0
    _check(inp, gpu, out_dtype=out_dtype)
    _check(inp, gpu, out_dtype=out_dtype, partition_size=256)


@pytest.mark.parametrize("out_dtype", [F32, BF])
@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("vs", [(2.0 ** 60, 2.0, 2.0 ** -56), (2.0 ** 60, 2.0, 2.0 ** -58), (1.0, 2.0 ** -59, 2.0 ** -118),
                                (2.0 ** -58, 2.0 ** 60, 2.0), (3e18, 7.0, 1e-17, 5e-36)])
def test_scales_that_fall_step_by_step(gpu, vs, hq, out_dtype):
    """Scales that fall from one stretch of a context to the next, each by less than 2^64, all with weight: the output is
    that of the large ones, and finite."""
    inp = decode_inputs(62, (128 * len(vs) * 2,), hq, 1, 16, BF)
    n = inp["block_tables"].shape[1]
    for i, b in enumerate(inp["block_tables"][0].tolist()):
        inp["v_scales"][b] = vs[i * len(vs) // n]
    for P in (0, 4096):                                               # (the second: one part, all falls in each warp)
        _check(inp, gpu, out_dtype=out_dtype, partition_size=P)


@pytest.mark.parametrize("out_dtype", [F32, BF])
@pytest.mark.parametrize("hq,bs", [(2, 16), (2, 32), (16, 16)])
@pytest.mark.parametrize("at", [0, 5, 14])
def test_heads_that_see_scales_far_apart(gpu, at, hq, bs, out_dtype):
    """Some heads have all their weight on a block of 2^64 times the others' scale, the others none: each is right."""
    inp = decode_inputs(63, (480,), hq, 1, bs, BF)
    b = int(inp["block_tables"][0, at])
    inp["q"][:] = inp["q"][:, :1].abs()
    inp["q"][:, 1::2] *= -1
    inp["k_cache"].view(torch.uint8)[b] &= 0x7F
    inp["k_scales"][b] = 2.0
    inp["v_scales"][:] = 2.0 ** -20
    inp["v_scales"][b] = 2.0 ** 44
    _check(inp, gpu, out_dtype=out_dtype)
    _check(inp, gpu, out_dtype=out_dtype, partition_size=160)


@pytest.mark.parametrize("out_dtype", [F32, BF])
@pytest.mark.parametrize("vs", [(2.0 ** -130, 0.0, 1.5 * 2.0 ** -130, -(2.0 ** -129)), (0.0, 2.0 ** -149, 2.0 ** -130),
                                (2.0 ** 118, 0.0, 1.7 * 2.0 ** 117), (2.0 ** -64, 2.0 ** -140, 0.0)])
def test_scales_at_the_ends_of_fp32(gpu, vs, out_dtype):
    """Scales without a finite reciprocal, zeros beside them, and scales near the largest number.  (Outputs stay above
    2^-126: the roundings of a few subnormal terms, 2^-150 each, are nothing beside 2^-20 of the values.)"""
    inp = decode_inputs(64, (400, 30), 4, 1, 16, BF)
    n = inp["v_scales"].shape[0]
    for b in range(n):
        inp["v_scales"][b] = vs[b % len(vs)]
    _check(inp, gpu, out_dtype=out_dtype)
    _check(inp, gpu, out_dtype=out_dtype, partition_size=64)


@pytest.mark.parametrize("factor", [1e-30, 1e-4, 20.0])
def test_small_and_large_queries(gpu, factor):
    inp = decode_inputs(5, (300, 40), 8, 2, 16, BF)
    inp["q"] = (inp["q"].float() * factor).to(BF)
    inp["q"][0, 3] = 0
    _check(inp, gpu)


def test_rising_scores(gpu):
    """Keys that grow along the context, so that the running reference is raised again and again, and then fall."""
    inp = decode_inputs(6, (1000,), 4, 1, 16, BF)
    bt = inp["block_tables"][0].long()
    up = torch.cat([torch.arange(40), torch.arange(40, 17, -1)]).float()[: len(bt)]
    inp["k_scales"][bt, 0] = torch.exp2(up / 4 - 12)
    _check(inp, gpu)
    _check(inp, gpu, partition_size=32)


def test_one_heavy_token_among_many_light_ones(gpu):
    inp = decode_inputs(8, (9000,), 4, 1, 16, BF, poison=False)
    inp["k_cache"].view(torch.uint8)[:] &= 0x87                      # small keys: subnormal e4m3 values
    inp["k_cache"].view(torch.uint8)[inp["block_tables"][0, 3].long(), :, 2] = 0x78
    _check(inp, gpu, scale=0.3)
    _check(inp, gpu, scale=0.3, partition_size=9008)


def test_long_sums_keep_their_size(gpu):
    """fp32 outputs of one part of 16384 tokens are not smaller than they should be: the products round towards zero,
    each of the 4 of a pair of units by less than 2^-23 of their sum, and nothing else rounds to one side."""
    inp = decode_inputs(90, (16384,), 8, 1, 16, BF)
    out = _check(inp, gpu, partition_size=16384)
    ref = decode_ref(inp, SCALE, F32)[0]
    size = (to64(out) * ref).sum() / (ref * ref).sum() - 1
    assert abs(size) <= 4 * 2.0 ** -23 + 2.0 ** -21      # (the second: 1024 outputs' own rounding, on average)


def test_length_one_is_the_scaled_value(gpu):
    inp = decode_inputs(9, (1, 1, 1), 4, 2, 16, BF)
    out = pkv.paged_attention_decode_fp8(**_dev(inp, gpu), scale=SCALE)
    for s in range(3):
        b = int(inp["block_tables"][s, 0])
        for h in range(4):
            want = inp["v_cache"][b, h // 2, 0].float() * inp["v_scales"][b, h // 2]
            assert torch.equal(out[s, h].cpu(), want)


def test_all_values_of_e4m3(gpu):
    """Every finite byte, as a key and as a value."""
    inp = decode_inputs(10, (256,), 4, 1, 16, FP)
    every = torch.tensor([b for b in range(256) if b & 0x7F != 0x7F], dtype=torch.uint8)
    n = inp["k_cache"].numel()
    inp["v_cache"] = every.repeat(-(-n // 254))[:n].view(torch.float8_e4m3fn).view(inp["v_cache"].shape)
    inp["k_cache"] = every.flip(0).repeat(-(-n // 254))[:n].view(torch.float8_e4m3fn).view(inp["k_cache"].shape)
    _check(inp, gpu, scale=0.002)


def test_nan_in_the_context_comes_through(gpu):
    """A NaN among the attended keys or values is not lost, with one partition or many; other rows are not touched."""
    for P in (0, 64, 16):
        for which in ("k_cache", "v_cache"):
            inp = decode_inputs(11, (400, 300), 8, 2, 16, BF)
            b = int(inp["block_tables"][0, 4])
            inp[which].view(torch.uint8)[b, 1, 3, 77] = 0x7F
            out = pkv.paged_attention_decode_fp8(**_dev(inp, gpu), scale=SCALE, partition_size=P)
            bad = out[0, 4:]
            assert (bad.isnan().all() if which == "k_cache" else bad[:, 77].isnan().all()), (P, which)
            assert not out[0, :4].isnan().any() and not out[1].isnan().any()


def test_queries_that_are_not_finite(gpu):
    """A head whose query holds a NaN or an infinity is NaN; the other heads of its group are not touched."""
    for bad in (math.nan, math.inf, -math.inf):
        for P in (0, 64, 16):
            inp = decode_inputs(25, (400, 30), 8, 2, 16, BF)
            clean = pkv.paged_attention_decode_fp8(**_dev(inp, gpu), scale=SCALE, partition_size=P)
            inp["q"][0, 5, 17] = bad
            out = pkv.paged_attention_decode_fp8(**_dev(inp, gpu), scale=SCALE, partition_size=P)
            assert out[0, 5].isnan().all()
            keep = torch.ones(2, 8, dtype=torch.bool)
            keep[0, 5] = False
            assert torch.equal(out.cpu()[keep], clean.cpu()[keep])


@pytest.mark.parametrize("scale", [0.0, -SCALE, 2.0])
def test_softmax_scales(gpu, scale):
    _check(decode_inputs(26, (300, 17), 8, 2, 32, FP), gpu, scale=scale)
    _check(decode_inputs(26, (300, 17), 8, 2, 32, FP), gpu, scale=scale, partition_size=32)


def test_tables_wider_than_the_contexts(gpu):
    """max_context_len far above the lengths: most partitions have nothing, entries past a context are never read."""
    inp = decode_inputs(27, (40, 700, 0), 8, 2, 16, BF)
    wide = torch.full((3, 2000), 2 ** 31 - 1, dtype=torch.int32)
    for s, L in enumerate((40, 700, 0)):
        n = -(-L // 16)
        wide[s, :n] = inp["block_tables"][s, :n]
    ref = _check(inp, gpu, partition_size=512)
    out = pkv.paged_attention_decode_fp8(**{**_dev(inp, gpu), "block_tables": wide.to(gpu)}, scale=SCALE,
                                         partition_size=512)
    assert pkv.check_device_error() == 0
    assert (out - ref).abs().max().item() <= 2.0 ** -18    # merged by the other kernel: another order of sums
    _check({**inp, "block_tables": wide}, gpu)


def test_physical_order_is_invisible(gpu):
    a = decode_inputs(12, (700, 90, 333), 8, 2, 16, BF)
    nb = a["k_cache"].shape[0]
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(1))
    b = dict(a)
    for x in ("k_cache", "v_cache", "k_scales", "v_scales"):
        t = a[x].view(torch.uint8) if a[x].dtype == torch.float8_e4m3fn else a[x]
        b[x] = torch.empty_like(t)
        b[x][perm] = t
        b[x] = b[x].view(a[x].dtype)
    b["block_tables"] = torch.where(a["block_tables"] >= 0, perm[a["block_tables"].clamp(min=0).long()].int(), -1)
    for P in (0, 64):
        x, y = (pkv.paged_attention_decode_fp8(**_dev(i, gpu), scale=SCALE, partition_size=P) for i in (a, b))
        assert torch.equal(x, y)


def test_bad_metadata_is_reported_and_zeroed(gpu):
    pkv.check_device_error()
    inp = decode_inputs(13, (300, 900, 100), 8, 2, 16, BF)
    nb = inp["k_cache"].shape[0]
    for P in (0, 64, 16):
        for bad in (nb, -1, 2 ** 31 - 1, -(2 ** 31)):
            d = _dev(inp, gpu)
            d["block_tables"][1, 3] = bad
            out = pkv.paged_attention_decode_fp8(**d, scale=SCALE, partition_size=P)
            assert pkv.check_device_error() == 4
            assert not out[1].any() and out[0].any() and out[2].any()
        for bad in (901, -1, 2 ** 31 - 1, -(2 ** 31)):
            d = _dev(inp, gpu)
            d["context_lens"][2] = bad
            out = pkv.paged_attention_decode_fp8(**d, scale=SCALE, partition_size=P, max_context_len=900)
            assert pkv.check_device_error() == 3
            assert not out[2].any() and out[0].any()


@pytest.mark.parametrize("P", [0, 64])
def test_workspace_with_anything_in_it(gpu, P):
    inp = _dev(decode_inputs(14, (1200, 2000, 0, 640), 8, 2, 16, BF), gpu)
    need = pkv.paged_attention_workspace_bytes(4, 8, 128, 2000, P)
    ws = torch.empty(need, dtype=torch.uint8, device=gpu)
    outs = []
    for fill in (0x00, 0xFF, 0x5A, None):
        if fill is not None:
            ws.fill_(fill)
        outs.append(pkv.paged_attention_decode_fp8(**inp, scale=SCALE, max_context_len=2000, partition_size=P, workspace=ws))
    assert all(torch.equal(o, outs[0]) for o in outs[1:])
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_attention_decode_fp8(**inp, scale=SCALE, max_context_len=2000, partition_size=P, workspace=ws[:256])


def test_workspace_shared_by_two_graphs_and_the_16_bit_call(gpu):
    """Two captured calls of different sizes and an eager 16-bit call take turns on one workspace."""
    a = _dev(decode_inputs(15, (1200, 2000), 8, 2, 16, BF), gpu)
    b = _dev(decode_inputs(16, (900, 1, 1700), 8, 2, 32, BF), gpu)
    ws = torch.empty(pkv.paged_attention_workspace_bytes(3, 8, 128, 2048, 64), dtype=torch.uint8, device=gpu)
    kw = dict(scale=SCALE, partition_size=256, workspace=ws)    # max_context_len: what the tables hold
    kb = torch.randn(126, 2, 16, 128, device=gpu).to(BF)
    bt16 = torch.arange(126, dtype=torch.int32, device=gpu)[None]
    eager = lambda: pkv.paged_attention_decode(a["q"][:1], kb, kb, bt16, a["context_lens"][1:], **kw)
    ra, rb, re = pkv.paged_attention_decode_fp8(**a, **kw), pkv.paged_attention_decode_fp8(**b, **kw), eager()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in (a, b):
        g, o = torch.cuda.CUDAGraph(), torch.empty_like(x["q"], dtype=F32)
        with torch.cuda.graph(g):
            pkv.paged_attention_decode_fp8(**x, out=o, **kw)
        graphs.append(g)
        outs.append(o)
    for i in (0, 1, 1, 0, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], (ra, rb)[i])
        assert torch.equal(eager(), re)
    assert pkv.check_device_error() == 0


def test_streams(gpu):
    inp = _dev(decode_inputs(18, (1200, 2000, 5), 8, 2, 16, BF), gpu)
    ref = pkv.paged_attention_decode_fp8(**inp, scale=SCALE)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [pkv.paged_attention_decode_fp8(**inp, scale=SCALE, stream=s if i % 2 else s.cuda_stream)
            for i in range(4) for s in streams]                        # calls at once, a workspace each
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_calls_on_two_streams_at_once(gpu):
    """Writes into two pools and split decodes of both, issued to two streams side by side, as alone."""
    lens = (1200, 900, 40, 1)
    ins = [_dev(decode_inputs(70 + i, lens, 8, 2, 16, BF), gpu) for i in range(2)]
    alone = [pkv.paged_attention_decode_fp8(**x, scale=SCALE, partition_size=128) for x in ins]
    slots, pos = runs_of_tokens(np.random.default_rng(5), [(0, 70), (16, 1), (3, 40)], 16, 12)
    cases = [Case(80 + i, 4, 2, 16, BF, 64, False, True, slots, pos, 12, fp8=True) for i in range(2)]
    rows = [c.to_dev(gpu) for c in cases]
    for d, c in zip(rows, cases):
        pkv.paged_kv_append_rope_fp8(**d)
    fresh = [[c.to_dev(gpu) for _ in range(6)] for c in cases]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(gpu) for _ in range(2)], [[], []]
    for r in range(6):
        for i, st in enumerate(streams):
            pkv.paged_kv_append_rope_fp8(**fresh[i][r], stream=st)
            outs[i].append(pkv.paged_attention_decode_fp8(**ins[i], scale=SCALE, partition_size=128, stream=st))
    torch.cuda.synchronize()
    assert pkv.check_device_error() == 0
    for i in range(2):
        for r in range(6):
            assert torch.equal(outs[i][r], alone[i])
            for n in ("q_out", "k_cache", "v_cache", "k_scales", "v_scales"):
                assert torch.equal(fresh[i][r][n].view(torch.uint8), rows[i][n].view(torch.uint8)), n


def test_blocks_past_4_gib(gpu):
    hkv, bs = 8, 16
    nb = (1 << 32) // (hkv * bs * 128) + 300
    inp = decode_inputs(19, (700, 30), 16, hkv, bs, BF, poison=False)
    ref = pkv.paged_attention_decode_fp8(**_dev(inp, gpu), scale=SCALE)
    n = inp["k_cache"].shape[0]
    d = _dev(inp, gpu)
    for x in ("k_cache", "v_cache", "k_scales", "v_scales"):
        t = d[x].view(torch.uint8) if "cache" in x else d[x]
        big = torch.zeros((nb,) + t.shape[1:], dtype=t.dtype, device=gpu)
        big[nb - n:] = t
        d[x] = big.view(d[x].dtype)
    d["block_tables"] = torch.where(d["block_tables"] >= 0, d["block_tables"] + (nb - n), -1).int()
    out = pkv.paged_attention_decode_fp8(**d, scale=SCALE)
    assert pkv.check_device_error() == 0 and torch.equal(out, ref)


def test_more_partitions_than_one_grid_dimension(gpu):
    """65,600 one-block partitions: 64 blocks repeated 1025 times weigh as the 64 blocks once."""
    inp = decode_inputs(20, (1024,), 4, 1, 16, BF)
    d = _dev(inp, gpu)
    d["block_tables"] = d["block_tables"].repeat(1, 1025).contiguous()
    d["context_lens"] = d["context_lens"] * 1025
    out = pkv.paged_attention_decode_fp8(**d, scale=SCALE, partition_size=16)
    assert pkv.check_device_error() == 0
    ref, tol = decode_ref(inp, SCALE, F32)
    # the merge adds 8,200 partials one after the other in each of 8 warps, to a sum and to a total
    v = to64(inp["v_cache"].float())
    top = np.abs(v[np.isfinite(v)]).max() * np.nanmax(to64(inp["v_scales"]))
    assert (np.abs(to64(out) - ref) <= tol + 2 * 8200 * 2.0 ** -24 * top).all()


def test_many_sequences(gpu):
    lens = np.random.default_rng(3).integers(0, 70, 3000).tolist()
    inp = decode_inputs(21, lens, 4, 1, 16, BF)
    _check(inp, gpu, heads=[2])


def test_no_sequences_and_refusals(gpu):
    inp = _dev(decode_inputs(22, (40, 20), 4, 2, 16, BF), gpu)
    empty = {**inp, "q": inp["q"][:0], "block_tables": inp["block_tables"][:0], "context_lens": inp["context_lens"][:0]}
    assert pkv.paged_attention_decode_fp8(**empty, scale=SCALE).shape == (0, 4, 128)
    launches = pkv.launch_count()
    bad = [dict(q=inp["q"][:1]), dict(q=inp["q"][..., :64].contiguous()), dict(k_scales=inp["k_scales"].half()),
           dict(v_scales=inp["v_scales"][:1]), dict(context_lens=inp["context_lens"].long()),
           dict(v_cache=inp["v_cache"][:1]), dict(block_tables=inp["block_tables"][0]), dict(q=inp["q"].cpu()),
           dict(k_scales=inp["k_scales"].t().contiguous().t()), dict(out=torch.empty(2, 3, 128, device=gpu))]
    for b in bad:
        with pytest.raises(ValueError):
            pkv.paged_attention_decode_fp8(**{**inp, **b}, scale=SCALE)
    for b in (dict(q=inp["q"].float()), dict(q=inp["q"][:, :3].contiguous()), dict(k_cache=inp["k_cache"].half(),
                                                                                 v_cache=inp["v_cache"].half())):
        with pytest.raises(pkv.PagedKVError):
            pkv.paged_attention_decode_fp8(**{**inp, **b}, scale=SCALE)
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_attention_decode_fp8(**inp, scale=SCALE, max_context_len=4096)   # above the tables' capacity
    assert pkv.launch_count() == launches


# ------------------------------------------------------------------ copies
@pytest.mark.parametrize("layers,hkv,bs", [(1, 8, 16), (3, 5, 32), (49, 1, 16), (2, 40, 32)])
def test_copy_blocks_fp8(gpu, layers, hkv, bs):
    """Bytes and scales of every layer (49: two launches), NaN bytes and scales among them; other blocks untouched."""
    rng = np.random.default_rng(layers)
    nb = 40
    pools = [[torch.from_numpy(rng.integers(0, 256, (nb, hkv, bs, D), dtype=np.uint8)) for _ in range(layers)] for _ in "kv"]
    scales = [[torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, (nb, hkv), dtype=np.int64).astype(np.int32))
               for _ in range(layers)] for _ in "kv"]
    perm = rng.permutation(nb)
    pairs = np.stack([np.append(perm[:16], perm[0]), perm[16:33]], axis=1).astype(np.int64)  # one source twice
    dp = [[t.to(gpu) for t in x] for x in pools]
    ds = [[t.to(gpu) for t in x] for x in scales]
    pkv.copy_blocks_fp8(*([t.view(torch.float8_e4m3fn) for t in x] for x in dp), *([t.view(F32) for t in x] for x in ds),
                        torch.from_numpy(pairs).to(gpu))
    assert pkv.check_device_error() == 0
    for host, dev in list(zip(pools, dp)) + list(zip(scales, ds)):
        for a, b in zip(host, dev):
            a[pairs[:, 1]] = a[pairs[:, 0]]
            assert torch.equal(a, b.cpu())


def test_copy_blocks_fp8_bad_ids_and_refusals(gpu):
    pkv.check_device_error()
    c = torch.zeros(6, 2, 16, D, dtype=torch.uint8, device=gpu)
    c[1] = 7
    k, s = c.view(torch.float8_e4m3fn), torch.arange(12.0, device=gpu).view(6, 2)
    for bad in ([0, 6], [6, 0], [-1, 2], [2, 1 << 40]):
        pkv.copy_blocks_fp8(k, k.clone(), s, s.clone(), torch.tensor([[1, 3], bad], device=gpu))
        assert pkv.check_device_error() == 2
        assert (c[3] == 7).all() and not c[0].any() and not c[2].any() and torch.equal(s[3], s[1])
    pkv.copy_blocks_fp8(k, k, s, s, torch.empty((0, 2), dtype=torch.int64, device=gpu))
    for a in ((k, k, s.double(), s), (k, k, s, s[:3]), (k, k[:3], s, s), ([k, k], [k], [s, s], [s, s])):
        with pytest.raises(ValueError):
            pkv.copy_blocks_fp8(*a, torch.tensor([[1, 3]], device=gpu))
    with pytest.raises(pkv.PagedKVError):
        pkv.copy_blocks_fp8(k.half(), k.half(), s, s, torch.tensor([[1, 3]], device=gpu))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("bs", [16, 32])
def test_a_forked_chat_on_an_8_bit_cache(gpu, bs):
    """A prompt in chunks, a fork, copy-on-write and decode steps: the attention of every step is attention over the
    values that the cache then stands for, and those are the 16-bit cache's within the rounding to e4m3."""
    g = torch.Generator().manual_seed(bs)
    hq, hkv, nb, prompt, steps = 8, 2, 40, 3 * bs + 5, bs + 4
    bm = pkv.BlockManager(nb, bs, np.random.default_rng(bs).permutation(nb))
    table = cos_sin_table(256, 64).to(gpu)
    k8, v8 = (torch.full((nb, hkv, bs, D), 0x7F, dtype=torch.uint8, device=gpu).view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.full((nb, hkv), math.nan, device=gpu) for _ in range(2))
    k16, v16 = (torch.full((nb, hkv, bs, D), math.nan, dtype=BF, device=gpu) for _ in range(2))
    w = torch.ones(D, dtype=BF, device=gpu)

    def write(slots, positions):
        n = len(slots)
        rows = torch.randn(n, hq + 2 * hkv, D, generator=g).to(BF).to(gpu)
        args = (rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], torch.tensor(positions, device=gpu), table,
                torch.tensor(slots, device=gpu))
        q8 = pkv.paged_kv_append_rope_fp8(*args, k8, v8, ks, vs, q_norm=w, k_norm=w)
        q = pkv.paged_kv_append_rope(*args, k16, v16, q_norm=w, k_norm=w)
        assert torch.equal(q8, q)
        return q

    def attend(q, seqs):
        bt = torch.full((len(seqs), nb), -1, dtype=torch.int32)
        for i, s in enumerate(seqs):
            ids = bm.block_table(s)
            bt[i, : len(ids)] = torch.tensor(ids)
        cl = torch.tensor([bm.num_tokens(s) for s in seqs], dtype=torch.int32)
        inp = dict(q=q, k_cache=k8, v_cache=v8, k_scales=ks, v_scales=vs, block_tables=bt, context_lens=cl)
        _check(inp, gpu, max_context_len=int(cl.max()))
        # a row was rounded once, and once more for each raise of its block's scale (3 of them would already be many)
        for i, L in enumerate(cl.tolist()):
            ids = bt[i, : -(-L // bs)].long().to(gpu)
            for c8, sc, c16 in ((k8, ks, k16), (v8, vs, v16)):
                a, b, step = c8[ids].float() * sc[ids][..., None, None], c16[ids].float(), sc[ids][..., None, None]
                a, b = (x.transpose(1, 2).flatten(0, 1)[:L] for x in (a, b))
                step = step.expand(-1, -1, bs, D).transpose(1, 2).flatten(0, 1)[:L]
                once = b.abs() * (2.0 ** -4 + 2.0 ** -8) + step * 2.0 ** -10
                assert ((a - b).abs() <= 4 * once).all()

    bm.add_sequence(0)
    for chunk in (bs + 3, prompt - bs - 3):
        p0 = bm.num_tokens(0)
        slots, _ = bm.append_tokens(0, chunk)
        write(list(slots), list(range(p0, p0 + chunk)))
    bm.fork(0, 1)
    for _ in range(steps):
        slots, pos, cows = [], [], []
        for s in (0, 1):
            pos.append(bm.num_tokens(s))
            slot, cow = bm.append_token(s)
            slots.append(slot)
            cows += [cow] if cow else []
        if cows:
            pairs = torch.tensor(cows, dtype=torch.int64, device=gpu)
            pkv.copy_blocks_fp8(k8, v8, ks, vs, pairs)
            pkv.copy_blocks(k16, v16, pairs)
        attend(write(slots, pos), [0, 1])
    assert pkv.check_device_error() == 0


def test_step_captured_in_one_graph(gpu):
    """Copy, rotating write and attention of a step in one graph, replayed, equal the calls made one by one."""
    inp = decode_inputs(31, (200, 77, 16), 8, 2, 16, BF, poison=False)
    slots = [int(inp["block_tables"][s, (L - 1) // 16]) * 16 + (L - 1) % 16 for s, L in enumerate((200, 77, 16))]
    c = Case(40, 8, 2, 16, BF, 128, False, True, slots, [199, 76, 15], inp["k_cache"].shape[0], fp8=True)

    def make():
        d, a = _dev(inp, gpu), c.to_dev(gpu)
        for x in ("k_cache", "v_cache", "k_scales", "v_scales"):
            a[x] = d[x]
        nb = d["k_cache"].shape[0]
        free = [b for b in range(nb) if b not in set(inp["block_tables"].flatten().tolist())]
        pairs = torch.tensor([[int(inp["block_tables"][0, 0]), free[0]]], device=gpu)
        return d, a, pairs, torch.empty(3, 8, D, device=gpu)

    def step(d, a, pairs, out):
        pkv.copy_blocks_fp8(d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"], pairs)
        q = pkv.paged_kv_append_rope_fp8(**a)
        pkv.paged_attention_decode_fp8(**{**d, "q": q}, scale=SCALE, out=out, max_context_len=200)

    one, two = make(), make()
    step(*one)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*two)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(one[3], two[3]) and torch.equal(one[1]["q_out"], two[1]["q_out"])
    for x in ("k_cache", "v_cache"):
        assert torch.equal(one[0][x].view(torch.uint8), two[0][x].view(torch.uint8))
    for x in ("k_scales", "v_scales"):
        assert torch.equal(one[0][x], two[0][x])
    assert pkv.check_device_error() == 0
