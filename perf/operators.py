"""Workloads of the rotating cache writes and the 8-bit cache: what is timed and compared.

Four operators, all on a paged cache [num_blocks, num_kv_heads, block_size, 128]:

* ``rope``    -- new queries, keys and values of a step: optional RMS norm of every query and key head, rotation by
  position, keys and values into their slots of a 16-bit cache.
* ``rope8``   -- the same into an e4m3 cache that holds one fp32 scale for each (block, KV head).
* ``decode8`` -- decode attention over such an e4m3 cache.
* ``copy8``   -- copy-on-write copies of blocks of such a cache, scales included, over several layers.

``run`` computes each in plain torch operations, in 32 bits, or, where ``own`` is true, through this package's calls.
Sizes are those of the package's workloads (32/8 heads and 64 sequences; 64/8 heads and 131072 tokens; 40/40 heads;
forked prompts; a four-sequence batch) and odd ones between them.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128                 # head dimension of every cache
E4M3_MAX = 448.0
MAX_POSITION = 131072   # rows of the rotation table
BASE = 500000.0         # rotation base
EPS = 1e-6
MIN_EXP = -64           # smallest scale of an e4m3 block: 2^-64

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token for each of 64 chats (32/8 heads): a decode step, where latency counts
        dict(name="rope step 64", op="rope", tokens=64, seqs=64, hq=32, hkv=8, bs=16, dtype="bf16", rot=128,
             interleaved=False, norm=False, padded=0),
        # a chunk of odd length from seven prompts, half of each head rotated in neighbouring pairs, padded batch
        dict(name="rope chunk 1537", op="rope", tokens=1537, seqs=7, hq=40, hkv=40, bs=16, dtype="fp16", rot=64,
             interleaved=True, norm=False, padded=23),
        # a long prompt's chunk with normed query and key heads (64/8 heads)
        dict(name="rope prefill 16384 normed", op="rope", tokens=16384, seqs=3, hq=64, hkv=8, bs=32, dtype="bf16",
             rot=128, interleaved=False, norm=True, padded=0),
        # one new token for each of 256 samples: rows join blocks that are partly filled
        dict(name="rope8 step 256", op="rope8", tokens=256, seqs=256, hq=32, hkv=8, bs=16, dtype="bf16", rot=128,
             interleaved=False, norm=False, padded=0),
        # ragged chunk, 40 heads, normed, padded batch
        dict(name="rope8 chunk 777", op="rope8", tokens=777, seqs=5, hq=40, hkv=40, bs=32, dtype="fp16", rot=64,
             interleaved=True, norm=True, padded=9),
        # many prompts written in one call
        dict(name="rope8 prefill 16384", op="rope8", tokens=16384, seqs=41, hq=32, hkv=8, bs=16, dtype="bf16", rot=128,
             interleaved=False, norm=False, padded=0),
        # four short chats: the smallest step
        dict(name="decode8 tiny", op="decode8", seqs=4, lo=1, hi=100, hq=4, hkv=1, bs=16, dtype="bf16", out="fp32"),
        # 64 chats of 512 to 4096 tokens, 32/8 heads
        dict(name="decode8 64x4096", op="decode8", seqs=64, lo=512, hi=4096, hq=32, hkv=8, bs=16, dtype="bf16",
             out="fp32"),
        # 128 chats of up to 2048 tokens without shared KV heads, some rows of the batch empty
        dict(name="decode8 128x2048 mha", op="decode8", seqs=128, lo=0, hi=2048, hq=40, hkv=40, bs=16, dtype="fp16",
             out="fp16"),
        # eight documents of 131072 tokens, 64/8 heads
        dict(name="decode8 8x131072", op="decode8", seqs=8, lo=131072, hi=131072, hq=64, hkv=8, bs=32, dtype="bf16",
             out="bf16"),
        # the first new tokens of 16 groups of 16 samples: 240 copies in one layer
        dict(name="copy8 240", op="copy8", pairs=240, layers=1, hkv=8, bs=16),
        # a fork's last block in every layer of a 40-layer model without shared KV heads
        dict(name="copy8 16x40", op="copy8", pairs=16, layers=40, hkv=40, bs=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope8", "decode8", "decode8", "copy8"])
    hq, hkv = rng.choice([(32, 8), (64, 8), (40, 40), (4, 1), (24, 3), (16, 1), (12, 2), (32, 1), (7, 7)])
    bs = rng.choice([16, 32])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "copy8":
        return dict(op=op, pairs=_log_int(rng, 1, 240), layers=rng.choice([1, 2, 3, 32, 33, 40]), hkv=min(hkv, 8), bs=bs)
    if op == "decode8":
        seqs = _log_int(rng, 1, 128)
        hi = _log_int(rng, 1, min(131072, max(64, 4000000 // (seqs * hkv))))
        lo = rng.choice([0, 1, hi // 8, hi])
        return dict(op=op, seqs=seqs, lo=lo, hi=hi, hq=hq, hkv=hkv, bs=bs, dtype=dtype,
                    out=rng.choice(["fp32", "bf16", "fp16"]))
    tokens = _log_int(rng, 1, 1200000 // (hq + 2 * hkv))
    tokens = min(tokens, 16384)
    seqs = tokens if rng.random() < 0.3 else _log_int(rng, 1, max(1, tokens // 8))
    return dict(op=op, tokens=tokens, seqs=seqs, hq=hq, hkv=hkv, bs=bs, dtype=dtype, rot=rng.choice([128, 128, 64, 32, 16, 0]),
                interleaved=rng.random() < 0.3, norm=rng.random() < 0.5, padded=rng.choice([0, 0, 1, 13]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _table(rot):
    """cos and sin of every position, [MAX_POSITION, rot]: cosines of the rot / 2 angles, then sines."""
    if rot == 0:
        return None
    inv = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(MAX_POSITION, dtype=torch.float64, device="cuda")[:, None] * inv[None, :]
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _pool8(g, nb, hkv, bs):
    """An e4m3 pool as earlier steps left it: values that fill their scales' range, scales of a few powers of two."""
    values = (_randn(g, nb, hkv, bs, D) * 110.0).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    e = torch.randint(-8, -5, (nb, hkv), generator=g, device="cuda")
    return values, torch.exp2(e.float())


def _append_inputs(case, seed):
    """One call's new tokens: sequences that start at a position of their own (inside a block, mostly) and run on, one
    after the other; `padded` rows behind them have no slot."""
    host, g = random.Random(seed), _gen(seed)
    T, S, bs, hq, hkv = case["tokens"], case["seqs"], case["bs"], case["hq"], case["hkv"]
    if S == T:
        counts = [1] * T
    else:
        cuts = sorted(host.sample(range(1, T), S - 1)) if S > 1 else []
        counts = [b - a for a, b in zip([0] + cuts, cuts + [T])]
    starts = [host.randrange(0, MAX_POSITION - n + 1) if host.random() < 0.8 else 0 for n in counts]
    first, nblocks = [], 0   # index of each sequence's first touched block
    for p, n in zip(starts, counts):
        first.append(nblocks - p // bs)
        nblocks += (p + n - 1) // bs - p // bs + 1
    most = T if S == T else T // bs + 2 * S   # blocks that such a call can touch
    nb = most + most // 4 + 1
    perm = torch.randperm(nb, generator=g, device="cuda")
    cnt = np.asarray(counts)
    pos = np.repeat(np.asarray(starts) - (np.cumsum(cnt) - cnt), cnt) + np.arange(T)
    logical = torch.from_numpy(pos // bs + np.repeat(np.asarray(first), cnt)).cuda()
    pos = torch.from_numpy(pos).cuda()
    slots = perm[logical] * bs + pos % bs
    pad = torch.full((case["padded"],), -1, dtype=torch.int64, device="cuda")
    rows = T + case["padded"]
    dt = TYPES[case["dtype"]]
    # the rows of one fused projection: queries, keys and values of a token side by side
    qkv = _randn(g, rows, hq + 2 * hkv, D)
    qkv[:, hq:hq + hkv] *= torch.exp(0.5 * _randn(g, hkv, D))  # some key channels are larger, as in trained models
    qkv = qkv.to(dt)
    st = dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], cos_sin=_table(case["rot"]),
              positions=torch.cat([pos, torch.zeros_like(pad)]), slots=torch.cat([slots, pad]),
              live=torch.arange(T, device="cuda"), blocks=perm[:nblocks].clone(),
              q_out=torch.zeros(rows, hq, D, dtype=dt, device="cuda"), q_norm=None, k_norm=None)
    if case["norm"]:
        st["q_norm"] = (1.0 + 0.1 * _randn(g, D)).to(dt)
        st["k_norm"] = (1.0 + 0.1 * _randn(g, D)).to(dt)
    if case["op"] == "rope":
        st["k_cache"], st["v_cache"] = _randn(g, nb, hkv, bs, D).to(dt), _randn(g, nb, hkv, bs, D).to(dt)
    else:
        st["k_cache"], st["k_scales"] = _pool8(g, nb, hkv, bs)
        st["v_cache"], st["v_scales"] = _pool8(g, nb, hkv, bs)
    return st


def _decode_inputs(case, seed):
    host, g = random.Random(seed), _gen(seed)
    B, bs, hq, hkv = case["seqs"], case["bs"], case["hq"], case["hkv"]
    lens = [host.randint(case["lo"], case["hi"]) for _ in range(B)]
    lens[host.randrange(B)] = case["hi"]
    n = [-(-L // bs) for L in lens]
    used = sum(n)
    nb = used + used // 8 + 1
    perm = torch.randperm(nb, generator=g, device="cuda").int()
    width = max(1, max(n))
    nn = torch.tensor(n, device="cuda")
    j = torch.arange(width, device="cuda")[None, :] + (nn.cumsum(0) - nn)[:, None]
    inside = torch.arange(width, device="cuda")[None, :] < nn[:, None]
    bt = torch.where(inside, perm[j.clamp(max=nb - 1)], -1).int().contiguous()
    k, ks = _pool8(g, nb, hkv, bs)
    v, vs = _pool8(g, nb, hkv, bs)
    return dict(case=case, q=_randn(g, B, hq, D).to(TYPES[case["dtype"]]), k_cache=k, v_cache=v, k_scales=ks, v_scales=vs,
                block_tables=bt, context_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), max_len=max(lens),
                scale=D ** -0.5)


def _copy_inputs(case, seed):
    g = _gen(seed)
    n, bs, hkv = case["pairs"], case["bs"], case["hkv"]
    nb = 2 * n + n // 4 + 1
    n_layers = case["layers"]
    (k, ks), (v, vs) = (_pool8(g, n_layers * nb, hkv, bs) for _ in range(2))
    perm = torch.randperm(nb, generator=g, device="cuda")
    st = dict(case=case, k=k.view(n_layers, nb, hkv, bs, D), v=v.view(n_layers, nb, hkv, bs, D),
              ks=ks.view(n_layers, nb, hkv), vs=vs.view(n_layers, nb, hkv),
              pairs=torch.stack([perm[:n], perm[n:2 * n]], dim=1).contiguous())
    st["layers"] = [[st[x][i] for i in range(n_layers)] for x in ("k", "v", "ks", "vs")]  # the model's caches
    return st


def prepare(case, seed):
    if case["op"] == "decode8":
        return _decode_inputs(case, seed)
    if case["op"] == "copy8":
        return _copy_inputs(case, seed)
    return _append_inputs(case, seed)


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return {"rope": _own_rope, "rope8": _own_rope8, "decode8": _own_decode8, "copy8": _own_copy8}[op](st)
    return {"rope": _rope, "rope8": _rope8, "decode8": _decode8, "copy8": _copy8}[op](st)


def _own_rope(st):
    import paged_kv_cache_11_gb300 as pkv
    q = pkv.paged_kv_append_rope(st["q"], st["k"], st["v"], st["positions"], st["cos_sin"], st["slots"], st["k_cache"],
                                 st["v_cache"], q_norm=st["q_norm"], k_norm=st["k_norm"], norm_eps=EPS,
                                 interleaved=st["case"]["interleaved"], q_out=st["q_out"])
    return dict(q=q, k_cache=st["k_cache"], v_cache=st["v_cache"])


def _own_rope8(st):
    import paged_kv_cache_11_gb300 as pkv
    q = pkv.paged_kv_append_rope_fp8(st["q"], st["k"], st["v"], st["positions"], st["cos_sin"], st["slots"],
                                     st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"], q_norm=st["q_norm"],
                                     k_norm=st["k_norm"], norm_eps=EPS, interleaved=st["case"]["interleaved"],
                                     q_out=st["q_out"])
    return dict(q=q, k_cache=st["k_cache"], v_cache=st["v_cache"], k_scales=st["k_scales"], v_scales=st["v_scales"])


def _own_decode8(st):
    import paged_kv_cache_11_gb300 as pkv
    return pkv.paged_attention_decode_fp8(st["q"], st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"],
                                          st["block_tables"], st["context_lens"], st["scale"],
                                          max_context_len=st["max_len"], out_dtype=TYPES[st["case"]["out"]])


def _own_copy8(st):
    import paged_kv_cache_11_gb300 as pkv
    pkv.copy_blocks_fp8(*st["layers"], st["pairs"])
    return [st["k"], st["v"], st["ks"], st["vs"]]


# the plain forms
def _normed(x, w):
    """x [T, H, D] in 32 bits, its heads divided by their root mean square and weighted."""
    return x if w is None else x / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * w.float()


def _rotated(x, table, positions, interleaved):
    if table is None:
        return x
    rot = table.shape[1]
    row = table[positions][:, None, :]
    c, s = row[..., : rot // 2], row[..., rot // 2:]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _new_rows(st):
    """The live tokens' rotated queries and keys and their values, in 32 bits, and their slots."""
    n = st["live"].numel()
    pos, inter = st["positions"][:n], st["case"]["interleaved"]
    q = _rotated(_normed(st["q"][:n].float(), st["q_norm"]), st["cos_sin"], pos, inter)
    k = _rotated(_normed(st["k"][:n].float(), st["k_norm"]), st["cos_sin"], pos, inter)
    return q, k, st["v"][:n].float(), st["slots"][:n]


def _rope(st):
    q, k, v, slots = _new_rows(st)
    bs, dt = st["case"]["bs"], st["q"].dtype
    st["q_out"][: q.shape[0]] = q.to(dt)
    at = (slots // bs, slice(None), slots % bs)
    st["k_cache"][at] = k.to(dt)
    st["v_cache"][at] = v.to(dt)
    return dict(q=st["q_out"], k_cache=st["k_cache"], v_cache=st["v_cache"])


def _power_scale(a):
    """The smallest power of two that brings a to 448 or less, 2^-64 at least."""
    m, e = torch.frexp(a)   # a = m 2^e, m in [1/2, 1): 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.exp2(torch.where(a > 0, e, MIN_EXP).clamp(min=MIN_EXP).float())


def _write8(cache, scales, rows, slots, blocks, bs):
    nb, hkv = scales.shape
    blk, off = slots // bs, slots % bs
    amax = torch.zeros(nb, hkv, device=rows.device)
    amax.scatter_reduce_(0, blk[:, None].expand(-1, hkv), rows.abs().amax(dim=-1), "amax")
    low = torch.full((nb,), bs, device=rows.device, dtype=torch.int64).scatter_reduce_(0, blk, off, "amin")
    a, low, old = amax[blocks], low[blocks][:, None], scales[blocks]
    new = torch.where((low > 0) & (a <= E4M3_MAX * old), old, _power_scale(a))
    # rows held below the first new one move to the new scale
    held = torch.arange(bs, device=rows.device)[None, :] < low
    tile = cache[blocks].float()
    moved = (tile * (old / new)[:, :, None, None]).to(torch.float8_e4m3fn)
    raw = cache.view(torch.uint8)
    raw[blocks] = torch.where(held[:, None, :, None], moved.view(torch.uint8), raw[blocks])
    scales[blocks] = new
    raw[blk, :, off] = (rows / scales[blk][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _rope8(st):
    q, k, v, slots = _new_rows(st)
    st["q_out"][: q.shape[0]] = q.to(st["q"].dtype)
    _write8(st["k_cache"], st["k_scales"], k, slots, st["blocks"], st["case"]["bs"])
    _write8(st["v_cache"], st["v_scales"], v, slots, st["blocks"], st["case"]["bs"])
    # an e4m3 tensor compares by its numbers; the scales beside it are the rest of each value
    return dict(q=st["q_out"], k_cache=st["k_cache"], v_cache=st["v_cache"], k_scales=st["k_scales"],
                v_scales=st["v_scales"])


def _gathered(cache, scales, ids):
    """[B, Hkv, tokens, D] in 32 bits: the blocks of every sequence, one after the other."""
    x = cache.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * scales[ids][..., None, None]
    B, n, hkv, bs, d = x.shape
    return x.transpose(1, 2).reshape(B, hkv, n * bs, d)


def _decode8(st):
    B, hq, _ = st["q"].shape
    hkv = st["k_cache"].shape[1]
    lens, ids = st["context_lens"], st["block_tables"].long().clamp(min=0)
    k, v = _gathered(st["k_cache"], st["k_scales"], ids), _gathered(st["v_cache"], st["v_scales"], ids)
    inside = (torch.arange(k.shape[2], device=k.device)[None, :] < lens[:, None])[:, None, None, :]
    q = st["q"].float().view(B, hkv, hq // hkv, D)
    s = torch.matmul(q, k.transpose(2, 3)) * st["scale"]
    s = torch.where(inside, s, -math.inf)
    m = s.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s - m)
    total = p.sum(dim=-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)
    o = torch.matmul(p, torch.where(inside.transpose(2, 3), v, 0.0))
    return o.reshape(B, hq, D).to(TYPES[st["case"]["out"]])


def _copy8(st):
    src, dst = st["pairs"][:, 0], st["pairs"][:, 1]
    k, v = st["k"].view(torch.uint8), st["v"].view(torch.uint8)
    k[:, dst], v[:, dst] = k[:, src], v[:, src]
    st["ks"][:, dst], st["vs"][:, dst] = st["ks"][:, src], st["vs"][:, src]
    return [st["k"], st["v"], st["ks"], st["vs"]]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "copy8":
        return dict(bytes=2 * 2 * case["pairs"] * case["layers"] * case["hkv"] * (case["bs"] * D + 4) + 16 * case["pairs"],
                    flops=0)
    hq, hkv, bs = case["hq"], case["hkv"], case["bs"]
    if op == "decode8":
        tokens = case["seqs"] * (case["lo"] + case["hi"]) / 2
        out = 4 if case["out"] == "fp32" else 2
        return dict(bytes=tokens * (hkv * 2 * D + (8 * hkv + 4) / bs) + case["seqs"] * (hq * D * (2 + out) + 4),
                    flops=4 * tokens * hq * D)
    T = case["tokens"]
    cache = 2 if case["op"] == "rope" else 1
    scales = 0 if case["op"] == "rope" else 2 * 4 * hkv * max(case["seqs"], T / bs)
    return dict(bytes=T * ((2 * hq + 2 * hkv) * D * 2 + 2 * hkv * D * cache + 4 * case["rot"] + 16) + scales,
                flops=T * (hq + hkv) * (3 * case["rot"] + (4 * D if case["norm"] else 0)))


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _turned64(x, w, table, positions, interleaved):
    x = x.double()
    if w is not None:
        x = x * (x.pow(2).sum(-1, keepdim=True) / D + EPS).rsqrt() * w.double()
    if table is None:
        return x
    rot = table.shape[1]
    t = table[positions].double()
    turn = torch.complex(t[:, : rot // 2], t[:, rot // 2:])[:, None, :]
    head = x[..., :rot]
    if interleaved:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * turn
        head = torch.view_as_real(z).reshape(head.shape)
    else:
        z = torch.complex(head[..., : rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn
        head = torch.cat([z.real, z.imag], dim=-1)
    return torch.cat([head, x[..., rot:]], dim=-1)


def _e4m3_64(x):
    """The e4m3 number nearest to x (ties to the even one): steps of 2^(e-3), e the exponent of x and -6 at least."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "copy8":
        return _copied_exact(st)
    if case["op"] == "decode8":
        return _attended_exact(st)
    n, bs, inter = case["tokens"], case["bs"], case["interleaved"]
    pos, slots = st["positions"][:n], st["slots"][:n]
    q = st["q_out"].double()
    q[:n] = _turned64(st["q"][:n], st["q_norm"], st["cos_sin"], pos, inter)
    rows = dict(k=_turned64(st["k"][:n], st["k_norm"], st["cos_sin"], pos, inter), v=st["v"][:n].double())
    got = dict(q=q)
    for x in ("k", "v"):
        cache = st[x + "_cache"].double()
        if case["op"] == "rope":
            cache[slots // bs, :, slots % bs] = rows[x]
        else:
            scales = st[x + "_scales"].double()
            _fill_exact(cache, scales, rows[x], slots, bs)
            got[x + "_scales"] = scales
        got[x + "_cache"] = cache
    return got


def _fill_exact(cache, scales, rows, slots, bs):
    """Block by block: sort the tokens by block, cut at the blocks' borders, all blocks of a cut at once."""
    order = torch.argsort(slots)
    rows, slots = rows[order], slots[order]
    blocks, which, counts = torch.unique_consecutive(slots // bs, return_inverse=True, return_counts=True)
    start = counts.cumsum(0) - counts
    first = slots[start] % bs
    top = torch.zeros(len(blocks), rows.shape[1], dtype=torch.float64, device=rows.device)
    for i in range(int(counts.max())):
        has = counts > i
        top[has] = torch.maximum(top[has], rows[start[has] + i].abs().amax(-1))
    old = scales[blocks]
    need = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)))  # may be one off at a power of two: mended below
    need = torch.where(need / 2 * E4M3_MAX >= top, need / 2, need)
    need = torch.where(need * E4M3_MAX < top, need * 2, need).clamp(min=2.0 ** MIN_EXP)
    new = torch.where((first[:, None] > 0) & (top <= old * E4M3_MAX), old, need)
    tile = cache[blocks]
    held = torch.arange(bs, device=rows.device)[None, None, :, None] < first[:, None, None, None]
    ratio = (old / new)[:, :, None, None]
    cache[blocks] = torch.where(held, _e4m3_64(tile * ratio), tile)
    scales[blocks] = new
    cache[slots // bs, :, slots % bs] = _e4m3_64(rows / new[which][:, :, None])


def _attended_exact(st):
    B, hq, _ = st["q"].shape
    hkv, bs = st["k_cache"].shape[1], st["k_cache"].shape[2]
    out = torch.zeros(B, hq, D, dtype=torch.float64, device="cuda")
    lens = st["context_lens"].tolist()
    for s, L in enumerate(lens):
        if L == 0:
            continue
        ids = st["block_tables"][s, : -(-L // bs)].long()
        k, v = (st[c].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * st[f][ids].double()[..., None, None]
                for c, f in (("k_cache", "k_scales"), ("v_cache", "v_scales")))
        k, v = (x.permute(1, 0, 2, 3).reshape(hkv, -1, D)[:, :L] for x in (k, v))
        z = torch.einsum("hgd,htd->hgt", st["q"][s].double().view(hkv, hq // hkv, D), k) * st["scale"]
        out[s] = torch.einsum("hgt,htd->hgd", torch.softmax(z, dim=-1), v).reshape(hq, D)
    return out


def _copied_exact(st):
    nb = st["k"].shape[1]
    origin = torch.arange(nb, device="cuda")  # the block whose contents each block has afterwards
    for src, dst in st["pairs"].tolist():
        origin[dst] = src
    return [x.double().index_select(1, origin) for x in (st["k"], st["v"], st["ks"], st["vs"])]
