"""The block write with rotation and norms, into 16-bit and e4m3 pools, against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_11_gb300 as pkv
from tests.fp8_helpers import Case, cos_sin_table, runs_of_tokens, to64

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def _run(case, gpu, expect=0, **kw):
    d = case.to_dev(gpu)
    d.update(kw)
    fn = pkv.paged_kv_append_rope_fp8 if case.fp8 else pkv.paged_kv_append_rope
    out = fn(**d)
    assert pkv.check_device_error() == expect
    return out, d


def _check(case, gpu, expect=0, **kw):
    out, d = _run(case, gpu, expect, **kw)
    if case.hq:
        case.check_q(out)
    if case.fp8:
        case.check_pools8(d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"])
    else:
        case.check_pools16(d["k_cache"], d["v_cache"])


SHAPES = [  # hq, hkv, bs, dtype, rot, interleaved, norm, fused
    (4, 1, 16, BF, 128, False, False, True),
    (8, 2, 32, FP, 128, True, True, True),
    (5, 5, 16, BF, 64, False, True, False),
    (3, 1, 32, FP, 16, True, False, True),
    (6, 2, 16, BF, 32, False, True, True),
    (2, 2, 16, FP, 112, False, False, False),
    (4, 4, 32, BF, 48, True, True, True),
    (4, 2, 16, BF, 0, False, True, True),
    (4, 2, 32, FP, 0, False, False, False),
    (0, 3, 16, BF, 128, False, True, True),
]
SPANS = [  # first position, tokens of each sequence
    [(0, 1)],
    [(0, 16), (5, 1), (31, 2)],
    [(3, 40), (0, 33), (15, 1), (16, 1), (14, 5)],
    [(0, 130)],
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("spans", range(len(SPANS)))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_shapes(gpu, shape, spans, fp8):
    hq, hkv, bs, dtype, rot, inter, norm, fused = SHAPES[shape]
    rng = np.random.default_rng(100 * shape + spans)
    slots, pos = runs_of_tokens(rng, SPANS[spans], bs, 24)
    _check(Case(7 * shape + spans, hq, hkv, bs, dtype, rot, inter, norm, slots, pos, 24, fused=fused, fp8=fp8), gpu)


@pytest.mark.parametrize("fp8", [False, True])
def test_one_token_for_each_of_many_sequences(gpu, fp8):
    rng = np.random.default_rng(5)
    slots, pos = runs_of_tokens(rng, [(int(p), 1) for p in rng.integers(0, 500, 70)], 16, 70)
    _check(Case(11, 8, 2, 16, BF, 128, False, False, slots, pos, 70, fp8=fp8), gpu)


@pytest.mark.parametrize("bs", [1, 7, 64])
def test_other_block_sizes_of_16_bit_pools(gpu, bs):
    rng = np.random.default_rng(bs)
    slots, pos = runs_of_tokens(rng, [(2, 20), (0, 3)], bs, 40)
    _check(Case(bs, 4, 2, bs, BF, 128, False, True, slots, pos, 40), gpu)


@pytest.mark.parametrize("fp8", [False, True])
def test_padding_between_and_around_the_tokens(gpu, fp8):
    """Padding rows keep their contents, and a block's run goes on behind padding, however much of it."""
    rng = np.random.default_rng(9)
    slots, pos = runs_of_tokens(rng, [(4, 9), (0, 20)], 16, 8)
    pad = lambda n: ([-1] * n, [-(1 << 40)] * n)  # the positions of padding are not read
    s2, p2 = pad(3)
    for i, (s, p) in enumerate(zip(slots, pos)):
        s2.append(s), p2.append(p)
        n = {2: 1, 3: 40, 6: 2, 15: 100}.get(i, 0)
        s2 += pad(n)[0]
        p2 += pad(n)[1]
    s2 += pad(70)[0]
    p2 += pad(70)[1]
    _check(Case(3, 4, 2, 16, BF, 128, False, True, s2, p2, 8, fp8=fp8), gpu)
    _check(Case(3, 4, 2, 16, BF, 128, False, True, [-1] * 5, [0] * 5, 8, fp8=fp8), gpu)   # nothing but padding


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_slots_and_positions(gpu, fp8):
    pkv.check_device_error()
    rng = np.random.default_rng(4)
    slots, pos = runs_of_tokens(rng, [(2, 14), (0, 6)], 16, 8)
    for i, code in ((0, 1), (5, 1), (13, 1), (19, 1)):      # a run's first, middle and last token
        s = list(slots)
        s[i] = 8 * 16 + 3 if i != 5 else 1 << 61
        _check(Case(i, 4, 2, 16, BF, 128, False, False, s, pos, 8, fp8=fp8), gpu, expect=code)
    for i, p in ((0, 512), (5, -1), (13, 1 << 62), (19, -(1 << 62))):
        ps = list(pos)
        ps[i] = p
        _check(Case(i, 4, 2, 16, BF, 128, False, False, slots, ps, 8, fp8=fp8), gpu, expect=8)
    ps = list(pos)
    ps[:14] = [-1] * 14                                     # a run of nothing but refused tokens
    _check(Case(1, 4, 2, 16, BF, 128, False, False, slots, ps, 8, fp8=fp8), gpu, expect=8)


def test_tokens_of_a_block_in_any_order(gpu):
    rng = np.random.default_rng(6)
    slots, pos = runs_of_tokens(rng, [(0, 16), (20, 11), (3, 4)], 16, 8)
    for a, b in ((0, 16), (16, 27), (27, 31)):
        o = a + rng.permutation(b - a)
        slots[a:b], pos[a:b] = [slots[i] for i in o], [pos[i] for i in o]
    _check(Case(2, 4, 2, 16, BF, 128, False, False, slots, pos, 8, fp8=True), gpu)


@pytest.mark.parametrize("grow", [1.0, 0.01, 60.0])
def test_joining_rows_keep_or_raise_the_scale(gpu, grow):
    """Rows that join a block: small ones leave its bytes and scale alone, large ones move them."""
    rng = np.random.default_rng(8)
    slots, pos = runs_of_tokens(rng, [(p, 2) for p in range(1, 14)], 16, 16)
    c = Case(21, 4, 2, 16, BF, 128, False, False, slots, pos, 16, fp8=True)
    c.rows.mul_(grow)
    _check(c, gpu)
    raw = c.kc.view(torch.uint8)
    raw[:, :, 0, :] = torch.arange(128, dtype=torch.uint8)          # every positive value and NaN among what moves
    raw[:, :, 2, :] = torch.arange(128, 256).to(torch.uint8)
    c.vc.view(torch.uint8)[:] = raw
    _check(c, gpu)


def test_scales_that_are_no_powers_of_two(gpu):
    rng = np.random.default_rng(8)
    slots, pos = runs_of_tokens(rng, [(p, 2) for p in (1, 5, 9, 14)], 16, 8)
    c = Case(22, 4, 2, 16, BF, 128, False, False, slots, pos, 8, fp8=True)
    c.ks.fill_(0.3)                                                   # large enough: kept
    c.vs.fill_(0.7)
    d = c.to_dev(gpu)
    pkv.paged_kv_append_rope_fp8(**d)
    assert torch.equal(d["k_scales"].cpu(), c.ks) and torch.equal(d["v_scales"].cpu(), c.vs)
    vals, sc = d["v_cache"].float().cpu(), 0.7
    for t, s in enumerate(slots):
        y = c.v[t].float()
        assert ((vals[s // 16, :, s % 16] * sc - y).abs() <= y.abs() * (2.0 ** -4 + 2.0 ** -20) + sc * 2.0 ** -10).all()


def test_unusable_scales_are_recorded_and_replaced(gpu):
    pkv.check_device_error()
    for bad in (float("nan"), 0.0, -1.0, float("inf"), -float("inf"), 2.0 ** -127):
        slots, pos = runs_of_tokens(np.random.default_rng(1), [(5, 3), (0, 4)], 16, 4)
        c = Case(23, 2, 1, 16, BF, 128, False, False, slots, pos, 4, fp8=True)
        c.ks.fill_(bad)
        _check(c, gpu, expect=9)
    c = Case(23, 2, 1, 16, BF, 128, False, False, slots[:3], pos[:3], 4, fp8=True)
    c.ks.fill_(2.0 ** -126)                                           # the smallest that counts: raised by the first row
    c.vs.fill_(2.0 ** -126)
    _check(c, gpu)
    c.rows.zero_()                                                    # and kept by rows of zeros
    _check(c, gpu)
    c = Case(23, 2, 1, 16, BF, 128, False, False, slots[3:], pos[3:], 4, fp8=True)
    c.ks.fill_(float("nan"))                                          # a fresh block never reads its scale
    c.vs.fill_(0.0)
    _check(c, gpu)


def test_values_at_the_ends_of_the_range(gpu):
    """Rows of zeros, the largest bf16 values, infinities and NaN; unrotated, so that every byte is exact."""
    slots, pos = runs_of_tokens(np.random.default_rng(1), [(0, 6), (16, 3), (32, 2), (48, 1), (64, 2)], 16, 8)
    c = Case(24, 2, 1, 16, BF, 0, False, False, slots, pos, 8, fused=False, fp8=True)
    c.k[0:6] = 0
    c.v[0:6, :, 5] = float("inf")
    c.v[3, :, 7:9] = float("nan")
    c.v[6:9] *= 1e38
    c.k[6, 0, 0] = 448.0 * 2.0 ** 20                                  # exactly what a power of two holds
    c.k[6:9, :, 1:] = 2.0 ** 12
    c.v[9:11] = float("-inf")                                         # no finite value at all
    c.k[9:11] *= 1e-30                                                # below the smallest scale's step: zeros
    c.k[11] = 448.0 * 2.0 ** -64
    c.v[12:14] = torch.finfo(BF).max
    _check(c, gpu)


def test_16_bit_values_at_the_ends_of_the_range(gpu):
    slots, pos = runs_of_tokens(np.random.default_rng(1), [(0, 4)], 16, 2)
    c = Case(25, 2, 1, 16, BF, 0, False, False, slots, pos, 2, fused=False)
    c.k[0], c.q[0] = float("inf"), float("-inf")
    c.v[1].view(torch.int16)[:] = 0x7FC1                              # a NaN's bits come through
    c.k[2], c.q[2] = 0, 0
    d = c.to_dev(gpu)
    out = pkv.paged_kv_append_rope(**d)
    for t, s in enumerate(slots):
        assert torch.equal(out[t].cpu(), c.q[t])
        assert torch.equal(d["k_cache"][s // 16, :, s % 16].cpu(), c.k[t])
        assert torch.equal(d["v_cache"][s // 16, :, s % 16].cpu().view(torch.int16), c.v[t].view(torch.int16))


@pytest.mark.parametrize("fp8", [False, True])
def test_queries_in_place_and_allocated(gpu, fp8):
    slots, pos = runs_of_tokens(np.random.default_rng(2), [(0, 20), (7, 3)], 16, 6)
    c = Case(26, 4, 2, 16, BF, 128, False, True, slots, pos, 6, fused=False, fp8=fp8)
    d = c.to_dev(gpu)
    d["q_out"] = d["q"]
    fn = pkv.paged_kv_append_rope_fp8 if fp8 else pkv.paged_kv_append_rope
    assert fn(**d) is d["q"]
    c.check_q(d["q"])
    out, _ = _run(c, gpu, q_out=None)
    c.check_q(out)


def test_broadcast_rows(gpu):
    """A token stride of zero: every token has the same rows."""
    slots, pos = runs_of_tokens(np.random.default_rng(2), [(0, 9)], 16, 2)
    c = Case(27, 4, 2, 16, BF, 128, False, False, slots, pos, 2, fused=False)
    for x in ("q", "k", "v"):
        setattr(c, x, getattr(c, x)[:1].expand(9, -1, -1))
    d = c.to_dev(gpu)
    for x in ("q", "k", "v"):
        d[x] = d[x][:1].contiguous().expand(9, -1, -1)
    c.check_q(pkv.paged_kv_append_rope(**d))
    c.check_pools16(d["k_cache"], d["v_cache"])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("which", ["q", "k"])
def test_one_of_the_norms(gpu, which, fp8):
    slots, pos = runs_of_tokens(np.random.default_rng(2), [(0, 20), (7, 3)], 16, 6)
    c = Case(34, 4, 2, 16, BF, 128, False, True, slots, pos, 6, fp8=fp8)
    setattr(c, "k_norm" if which == "q" else "q_norm", None)
    _check(c, gpu)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs", [16, 32])
def test_long_ragged_batches(gpu, bs, fp8):
    """Enough tokens for windows of 16 tokens and several heads per warp, with runs of every length and offset."""
    rng = np.random.default_rng(bs)
    spans = [(int(rng.integers(0, 60)), int(n)) for n in rng.integers(1, 3 * bs, 60)]
    slots, pos = runs_of_tokens(rng, spans, bs, 400)
    c = Case(35 + bs, 0, 3, bs, BF, 32, False, False, slots, pos, 400, fp8=fp8)
    _check(c, gpu)
    # many more tokens than the checked ones, in front of them: the same rows give the same bytes
    n, reps = len(slots), 8
    d = c.to_dev(gpu)
    big = {}
    for x in ("k", "v", "positions", "slot_mapping"):
        t = d[x]
        big[x] = torch.cat([t] * reps, dim=0) if x != "slot_mapping" else torch.cat(
            [t + i * 400 * bs for i in range(reps)])
    for x in ("k_cache", "v_cache", "k_scales", "v_scales"):
        if x in d:
            t = d[x].view(torch.uint8) if d[x].dtype == torch.float8_e4m3fn else d[x]
            big[x] = torch.cat([t] * reps, dim=0).view(d[x].dtype)
    fn = pkv.paged_kv_append_rope_fp8 if fp8 else pkv.paged_kv_append_rope
    fn(**{**d, **big})
    fn(**d)
    assert pkv.check_device_error() == 0 and n * reps > 8 * bs
    for x in ("k_cache", "v_cache", "k_scales", "v_scales"):
        if x in d:
            raw = (lambda t: t.view(torch.uint8) if t.element_size() == 1 else t)
            for i in range(reps):
                assert torch.equal(raw(big[x])[400 * i:400 * (i + 1)], raw(d[x])), (x, i)


@pytest.mark.parametrize("fp8", [False, True])
def test_far_positions(gpu, fp8):
    """Positions up to 131071: the angle is the table's, so nothing is lost on the way to them."""
    slots, _ = runs_of_tokens(np.random.default_rng(2), [(0, 8)], 16, 2)
    pos = [131071, 131070, 99999, 65536, 65535, 1, 0, 131071]
    _check(Case(28, 2, 1, 16, BF, 128, False, False, slots, pos, 2, max_position=131072, fp8=fp8), gpu)


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_past_4_gib(gpu, fp8):
    """Blocks at the far end of pools whose byte offsets need more than 32 bits."""
    hkv, bs = 8, 16
    nb = (1 << 32) // (hkv * bs * 128 * (1 if fp8 else 2)) + 200
    n = 40
    far = [nb - 1, nb - 100, nb - 7]
    slots = [far[t // bs] * bs + t % bs for t in range(n)]
    near = [t // bs * bs + t % bs for t in range(n)]
    got = []
    for blocks, s in ((nb, slots), (3, near)):
        c = Case(29, 2, hkv, bs, BF, 128, False, False, s, list(range(n)), 3, fp8=fp8)
        c.num_blocks = blocks
        d = c.to_dev(gpu)
        if blocks == nb:
            for x in ("k_cache", "v_cache"):
                d[x] = torch.zeros((nb, hkv, bs, 128), dtype=torch.uint8 if fp8 else BF, device=gpu)
                d[x] = d[x].view(torch.float8_e4m3fn) if fp8 else d[x]
            if fp8:
                d["k_scales"], d["v_scales"] = (torch.ones(nb, hkv, device=gpu) for _ in range(2))
        _run(c, gpu, **d)
        i = torch.tensor(far if blocks == nb else [0, 1, 2], device=gpu)
        rows = [d[x].view(torch.uint8)[i][:, :, :8].cpu() for x in ("k_cache", "v_cache")]
        got.append(rows + ([d["k_scales"][i].cpu(), d["v_scales"][i].cpu()] if fp8 else []))
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("fp8", [False, True])
def test_on_another_stream_and_captured(gpu, fp8):
    slots, pos = runs_of_tokens(np.random.default_rng(2), [(0, 30), (9, 1), (5, 2)], 16, 8)
    c = Case(30, 4, 2, 16, BF, 128, False, True, slots, pos, 8, fp8=fp8)
    fn = pkv.paged_kv_append_rope_fp8 if fp8 else pkv.paged_kv_append_rope
    s = torch.cuda.Stream()
    d = c.to_dev(gpu)
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        d["q_out"] = None
        out = fn(stream=stream, **d)
        s.synchronize()
        c.check_q(torch.where((d["slot_mapping"] < 0)[:, None, None], c.q_out.to(gpu), out))
    d = c.to_dev(gpu)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn(**d)
    start = {x: d[x].clone() for x in ("k_cache", "v_cache", "k_scales", "v_scales") if x in d}
    for _ in range(2):                                                # a replay takes what the pools hold then
        for x, t in start.items():
            d[x].copy_(t)
        g.replay()
        torch.cuda.synchronize()
        c.check_q(d["q_out"])
        if fp8:
            c.check_pools8(d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"])
        else:
            c.check_pools16(d["k_cache"], d["v_cache"])
    assert pkv.check_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_no_tokens(gpu, fp8):
    c = Case(31, 4, 2, 16, BF, 128, False, True, [], [], 4, fp8=fp8)
    launches = pkv.launch_count()
    _check(c, gpu)
    assert pkv.launch_count() == launches


def test_binding_refusals(gpu):
    slots, pos = runs_of_tokens(np.random.default_rng(2), [(0, 4)], 16, 2)
    c = Case(32, 4, 2, 16, BF, 128, False, True, slots, pos, 2, fp8=True)
    d = c.to_dev(gpu)
    launches = pkv.launch_count()
    bad = [dict(k=d["k"].float()), dict(k=d["k"][:3]), dict(v=d["v"][:, :1]), dict(q=d["q"].transpose(1, 2)),
           dict(slot_mapping=d["slot_mapping"].int()), dict(positions=None),
           dict(positions=d["positions"].int()), dict(cos_sin=d["cos_sin"].double()), dict(cos_sin=d["cos_sin"][:, :0]),
           dict(q_norm=d["q_norm"].float()), dict(k_norm=d["k_norm"][:64]), dict(q_out=d["q_out"][:, :1]), dict(q=None),
           dict(k_scales=d["k_scales"].half()), dict(v_scales=d["v_scales"].t()), dict(v_cache=d["v_cache"][:1]),
           dict(positions=d["positions"].cpu()), dict(q_out=d["q_out"].cpu())]
    for b in bad:
        with pytest.raises(ValueError):
            pkv.paged_kv_append_rope_fp8(**{**d, **b})
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_kv_append_rope_fp8(**{**d, "cos_sin": cos_sin_table(64, 24).to(gpu)})
    x = {k: v for k, v in d.items() if "scales" not in k}
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_kv_append_rope(**x)                                 # an e4m3 pool needs the other call
    assert pkv.launch_count() == launches


@pytest.mark.parametrize("fp8", [False, True])
def test_positions_without_a_table_are_not_read(gpu, fp8):
    slots, pos = runs_of_tokens(np.random.default_rng(4), [(0, 40), (3, 9)], 16, 8)
    c = Case(34, 4, 2, 16, FP, 0, False, True, slots, pos, 8, fp8=fp8)
    call = pkv.paged_kv_append_rope_fp8 if fp8 else pkv.paged_kv_append_rope
    names = ("q_out", "k_cache", "v_cache", "k_scales", "v_scales") if fp8 else ("q_out", "k_cache", "v_cache")
    a, b = c.to_dev(gpu), c.to_dev(gpu)
    far = torch.full((len(slots),), 1 << 62, device=gpu)
    call(**{**a, "positions": None, "cos_sin": None})
    call(**{**b, "positions": far, "cos_sin": None})
    for n in names:
        assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8))
    c.check_q(b["q_out"])
    pkv.check_device_error()


def test_the_plain_block_write_agrees(gpu):
    """Without rotation, norms and queries the call is paged_kv_append, bit for bit."""
    slots, pos = runs_of_tokens(np.random.default_rng(3), [(0, 50), (9, 4)], 16, 8)
    c = Case(33, 0, 3, 16, FP, 0, False, False, slots, pos, 8, fused=False)
    a, b = c.to_dev(gpu), c.to_dev(gpu)
    pkv.paged_kv_append_rope(**a)
    pkv.paged_kv_append(b["k"], b["v"], b["slot_mapping"], b["k_cache"], b["v_cache"])
    assert torch.equal(a["k_cache"], b["k_cache"]) and torch.equal(a["v_cache"], b["v_cache"])
    assert np.isfinite(to64(a["k_cache"])).all()


def _with_ends(c, kinds):
    """Puts rows at the ends of the range among c's (unfused) rows, a kind per token in turn."""
    for t in range(len(c.slots)):
        kind = kinds[t % len(kinds)]
        if kind == "zero":
            c.k[t], c.v[t] = 0, 0
        elif kind == "k inf":
            c.k[t, :, 3] = float("inf")
        elif kind == "v inf":
            c.v[t, 0, 126] = float("-inf")
        elif kind == "nan":
            c.k[t, :, ::2], c.v[t] = float("nan"), float("nan")
        elif kind == "large":
            c.k[t] *= 50.0
            c.v[t] *= 1e4
        elif kind == "small":
            c.k[t] *= 1e-3
            c.v[t] *= 1e-6


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("rot", [0, 64])
def test_steps_of_one_token(gpu, bs, rot, inter):
    """A token of each sequence, at every row of a block: joining rows that keep or raise the scale, infinities in
    the keys or the values alone, unusable scales."""
    rng = np.random.default_rng(bs + rot)
    spans = [(p % (2 * bs), 1) for p in range(3 * bs)]
    slots, pos = runs_of_tokens(rng, spans, bs, 4 * bs + 8)
    c = Case(41 + bs, 4, 3, bs, FP if inter else BF, rot, inter, False, slots, pos, 4 * bs + 8, fused=False, fp8=True)
    _check(c, gpu)
    c = Case(42 + bs, 4, 3, bs, BF, rot, inter, False, slots, pos, 4 * bs + 8, fused=False, fp8=True)
    _with_ends(c, ["", "large", "small", "zero", "nan"] + ([] if rot else ["k inf", "v inf"]))
    _check(c, gpu)
    pkv.check_device_error()
    c.ks[::3] = float("nan")
    c.vs[1::3] = 2.0 ** -127
    _check(c, gpu, expect=9)


def test_steps_of_one_token_with_norm(gpu):
    slots, pos = runs_of_tokens(np.random.default_rng(1), [(p, 1) for p in range(70)], 16, 400)
    _check(Case(43, 4, 3, 16, BF, 128, False, True, slots, pos, 400, fp8=True), gpu)


@pytest.mark.parametrize("hkv", [1, 3, 20])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("single", [False, True])
def test_runs_found_in_wide_windows(gpu, bs, hkv, single):
    """A checked batch repeated until a warp's window is a block and it has several heads: runs of every length, steps
    of one token, padding and rows with infinities among them give the bytes that the batch alone gives."""
    rng = np.random.default_rng(bs + hkv)
    lens = np.ones(40, dtype=int) if single else rng.choice([1, 1, 2, 7, bs - 1, bs, bs + 1, 3 * bs], 40)
    spans = [(int(rng.integers(0, 2 * bs)), int(n)) for n in lens]
    slots, pos = runs_of_tokens(rng, spans, bs, 240)
    for at, n in ((7, 3), (20, 1), (30, 50)):
        slots[at:at], pos[at:at] = [-1] * n, [0] * n
    c = Case(50 + hkv, 0, hkv, bs, BF, 0, False, False, slots, pos, 240, fused=False, fp8=True)
    _with_ends(c, [""] * 11 + ["k inf"] + [""] * 6 + ["v inf"])
    if hkv < 20:
        _check(c, gpu)
    d = c.to_dev(gpu)
    reps = -(-31 * 2 * 6080 // (hkv * len(slots)))
    big = {x: torch.cat([d[x]] * reps) for x in ("k", "v", "k_scales", "v_scales")}
    for x in ("k_cache", "v_cache"):
        big[x] = torch.cat([d[x].view(torch.uint8)] * reps).view(torch.float8_e4m3fn)
    s = d["slot_mapping"]
    big["slot_mapping"] = torch.cat([torch.where(s < 0, s, s + i * 240 * bs) for i in range(reps)])
    pkv.paged_kv_append_rope_fp8(**{**d, **big})
    pkv.paged_kv_append_rope_fp8(**d)
    assert pkv.check_device_error() == 0
    for x in ("k_cache", "v_cache", "k_scales", "v_scales"):
        one, all_ = (t.view(torch.uint8) if t.element_size() == 1 else t for t in (d[x], big[x]))
        assert (all_.view(reps, *one.shape) == one).all(), x


def _check_exact(c, gpu):
    """Keys that are neither turned nor normed and the same numbers as values: values are checked byte for byte (and the
    scales), keys have to be the same."""
    c.v, c.vc, c.vs = c.k.clone(), c.kc.clone(), c.ks.clone()
    _, d = _run(c, gpu)
    c.check_pools8(d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"])
    assert torch.equal(d["k_scales"], d["v_scales"])
    assert torch.equal(d["k_cache"].view(torch.uint8), d["v_cache"].view(torch.uint8))


@pytest.mark.parametrize("single", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("bs", [16, 32])
def test_rows_under_scales_that_are_no_powers_of_two_are_nearest(gpu, bs, dtype, single):
    """Rows that join a block whose scale is kept: the stored values are the nearest to y / scale, also where y / scale is
    next to the middle between two of them (scales are y / middle, rounded, for one y of the block)."""
    rng = np.random.default_rng(bs)
    blocks, hkv = 24, 3
    rows = [(p, 1) for p in range(1, blocks + 1)] if single else [(1 + b % 5, 2 + b % 11) for b in range(blocks)]
    slots, pos = [], []
    for b, (p, n) in enumerate(rows):
        p = 1 + (p - 1) % (bs - 1)
        for o in range(p, min(p + n, bs)):
            slots.append(b * bs + o), pos.append(o)
    c = Case(70, 0, hkv, bs, dtype, 0, False, False, slots, pos, blocks, fused=False, fp8=True)
    bits = 7 if dtype == BF else 10
    lowest = -100 if dtype == BF else -6
    for b in range(blocks):
        for h in range(hkv):
            y = (1 + int(rng.integers(0, 2 ** bits)) / 2 ** bits) * 2.0 ** int(rng.integers(lowest, 6))
            middle = (1 + (2 * int(rng.integers(0, 8)) + 1) / 16) * 2.0 ** int(rng.integers(-5, 7))
            c.ks[b, h] = [y / middle, 0.3 * 2.0 ** int(rng.integers(-3, 3)), 7.0 / 448, y / middle][(b + h) % 4]
            s = float(c.ks[b, h])
            for t in [t for t, x in enumerate(slots) if x // bs == b]:
                v = (1 + rng.integers(0, 2 ** bits, 128) / 2 ** bits) * 2.0 ** rng.integers(-11, 9, 128)
                v = np.minimum(v * 2.0 ** np.floor(np.log2(s)), min(400 * s, 6e4)) * rng.choice([-1, 1], 128)
                v[:8] = y * np.array([1, -1, 0.5, -0.5, 0.25, -2 if middle < 200 else 1, 1, 0])
                c.k[t, h] = torch.from_numpy(v).to(dtype)
    _check_exact(c, gpu)


@pytest.mark.parametrize("single", [False, True])
def test_rows_moved_from_a_scale_that_is_no_power_of_two(gpu, single):
    """Held values, every byte among them, go to the nearest of value * (old / new)."""
    n = 1 if single else 3
    slots = [b * 16 + 5 + o for b in range(40) for o in range(n)]
    c = Case(71, 0, 2, 16, BF, 0, False, False, slots, [0] * len(slots), 40, fused=False, fp8=True)
    raw = c.kc.view(torch.uint8)
    raw[:, :, 0, :] = torch.arange(128, dtype=torch.uint8)
    raw[:, :, 1, :] = torch.arange(128, 256).to(torch.uint8)
    rng = np.random.default_rng(3)
    for b in range(40):     # old / new = middle / value, rounded, for one value of the held ones
        value = (1 + int(rng.integers(0, 8)) / 8) * 2.0 ** int(rng.integers(-2, 8))
        middle = (1 + (2 * int(rng.integers(0, 8)) + 1) / 16) * 2.0 ** -3
        c.ks[b, :] = middle / value
        # (the new rows ask for a scale of 1, or a power of two more where the old one is large)
        c.k[[t for t, s in enumerate(slots) if s // 16 == b], 0] = 300.0
        c.k[[t for t, s in enumerate(slots) if s // 16 == b], 1] = 448.0
    _check_exact(c, gpu)


@pytest.mark.parametrize("single", [False, True])
def test_a_scale_is_kept_up_to_448_times_itself_exactly(gpu, single):
    """Rows just above what the old scale holds, by less than a 32-bit product 448 * scale can tell, raise it."""
    n = 1 if single else 2
    picks = []
    for m in range(128):
        a = np.float32((1 + m / 128) * 4.0)
        old = np.float32(float(a) / 448)
        if float(old) * 448 >= float(a):
            old = np.nextafter(old, np.float32(0))
        if np.float32(448) * old >= a:
            picks.append((float(a), float(old)))
    assert len(picks) >= 8
    slots = [b * 16 + 3 + o for b in range(len(picks)) for o in range(n)]
    c = Case(72, 0, 1, 16, BF, 0, False, False, slots, [0] * len(slots), len(picks), fused=False, fp8=True)
    for b, (a, old) in enumerate(picks):
        c.ks[b, 0] = old
        c.k[b * n:(b + 1) * n, 0] = 0.25
        c.k[b * n, 0, 7] = -a
    _check_exact(c, gpu)


@pytest.mark.parametrize("single", [False, True])
def test_kept_scales_at_the_ends_of_fp32(gpu, single):
    """The smallest and the largest scales that are kept, powers of two and not, with values down to subnormal ones."""
    n = 1 if single else 4
    scales = [2.0 ** -126, 1.3 * 2.0 ** -126, 1.9 * 2.0 ** -120, 2.0 ** 127, 1.9 * 2.0 ** 127, 1.1 * 2.0 ** 122]
    slots = [b * 16 + 2 + o for b in range(len(scales)) for o in range(n)]
    c = Case(73, 0, 2, 16, BF, 0, False, False, slots, [0] * len(slots), len(scales), fused=False, fp8=True)
    rng = np.random.default_rng(5)
    top = float(torch.finfo(BF).max)
    for b, s in enumerate(scales):
        c.ks[b] = s
        lo = -7 if s < 1 else -11
        v = (1 + rng.integers(0, 128, (n, 2, 128)) / 128) * 2.0 ** rng.integers(lo, 8, (n, 2, 128))
        c.k[b * n:(b + 1) * n] = torch.from_numpy(np.minimum(v * 2.0 ** np.floor(np.log2(s)), min(440 * s, top))).to(BF)
    _check_exact(c, gpu)
    c.k.neg_()
    _check_exact(c, gpu)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bs,hkv", [(16, 3), (16, 8), (32, 3), (32, 8)])
def test_turned_and_normed_keys_in_full_windows(gpu, bs, hkv, inter):
    """A checked batch of rotated and normed keys, repeated until the launch takes windows of a block less a token and four
    items (two heads) or more per warp, gives the bytes that the batch alone gives."""
    rng = np.random.default_rng(7 * bs + hkv)
    lens = rng.choice([1, 2, 7, bs - 1, bs, bs + 1, 3 * bs], 24)
    spans = [(int(rng.integers(0, 2 * bs)), int(n)) for n in lens]
    slots, pos = runs_of_tokens(rng, spans, bs, 160)
    for at, n in ((9, 2), (40, 1)):
        slots[at:at], pos[at:at] = [-1] * n, [0] * n
    c = Case(90 + hkv, 0, hkv, bs, FP if inter else BF, 64 if inter else 128, inter, True, slots, pos, 160, fp8=True)
    c.ks[::5] *= 1.3                                                  # (no powers of two)
    c.vs[::7] *= 1.7
    _check(c, gpu)
    d = c.to_dev(gpu)
    n, items, enough = len(slots), 4, {16: 4560, 32: 1520}[bs]
    groups = -(-2 * hkv // items)
    reps = -(-enough * (bs - 1) // (groups * n)) + 1
    assert n * reps // (bs - 1) * groups >= enough                    # what the launch asks for that window and 4 items
    big = {x: torch.cat([d[x]] * reps) for x in ("k", "v", "positions", "k_scales", "v_scales")}
    for x in ("k_cache", "v_cache"):
        big[x] = torch.cat([d[x].view(torch.uint8)] * reps).view(torch.float8_e4m3fn)
    s = d["slot_mapping"]
    big["slot_mapping"] = torch.cat([torch.where(s < 0, s, s + i * 160 * bs) for i in range(reps)])
    pkv.paged_kv_append_rope_fp8(**{**d, **big})
    pkv.paged_kv_append_rope_fp8(**d)
    assert pkv.check_device_error() == 0
    for x in ("k_cache", "v_cache", "k_scales", "v_scales"):
        one, all_ = (t.view(torch.uint8) if t.element_size() == 1 else t for t in (d[x], big[x]))
        assert (all_.view(reps, *one.shape) == one).all(), x
