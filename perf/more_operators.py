"""Workloads of drafted-token attention and of the latent cache: what is timed and compared.

Four operators:

* ``tree``    -- attention of several drafted tokens of each sequence, whose masks form a tree (or a chain), over a paged
  cache [num_blocks, num_kv_heads, block_size, 128].
* ``lwrite``  -- the write into a paged latent cache [num_blocks, block_size, 576]: RMS norm of each token's latent (512
  values), rotation by position of its key part (64 values) and of every query head's 64 values.
* ``latent``  -- attention over that cache in its absorbed form: every head's query has 576 values, and a token's first 512
  are its value too; one token of each sequence, or several drafted ones.
* ``prompt``  -- the expanded form for whole prompts: keys of 128 values a head beside 64 that the heads share, values of 128.

``run`` computes each in plain torch operations, in 32 bits, or, where ``own`` is true, through this package's calls.  Sizes
are those of the package's workloads (a four-sequence batch; 64 sequences of 512 to 4096 tokens; 40/40 heads and 128
sequences; 131072 tokens) and odd ones between them.
"""
import math
import random

import torch

own = False

D = 128                 # head dimension of the K/V cache, and of expanded keys and values
LATENT = 512            # values of a token's latent
ROT = 64                # rotated values beside it
ROW = LATENT + ROT
MAX_POSITION = 131072   # rows of the rotation table
BASE = 10000.0          # rotation base
EPS = 1e-6

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # four short chats, a tree of eight drafted tokens each: the smallest verify step
        dict(name="tree tiny", op="tree", seqs=4, lo=8, hi=100, n_lo=8, n_hi=8, hq=4, hkv=1, bs=16, dtype="bf16", tree=True),
        # 64 chats of 512 to 4096 tokens, 32/8 heads, trees of 16 drafted tokens
        dict(name="tree 64x4096 16", op="tree", seqs=64, lo=512, hi=4096, n_lo=16, n_hi=16, hq=32, hkv=8, bs=16,
             dtype="bf16", tree=True),
        # 128 chats without shared KV heads, chains of one to five drafted tokens, ragged
        dict(name="tree 128x2048 mha chain", op="tree", seqs=128, lo=5, hi=2048, n_lo=1, n_hi=5, hq=40, hkv=40, bs=16,
             dtype="fp16", tree=False),
        # eight documents of 131072 tokens, 64/8 heads, trees of 31 drafted tokens
        dict(name="tree 8x131072 31", op="tree", seqs=8, lo=131072, hi=131072, n_lo=31, n_hi=31, hq=64, hkv=8, bs=32,
             dtype="bf16", tree=True),
        # one new token for each of 64 chats: the write of a decode step, where latency counts
        dict(name="lwrite step 64", op="lwrite", tokens=64, seqs=64, heads=128, bs=16, dtype="bf16", interleaved=True,
             norm=True, padded=0, copy=False),
        # many prompts' chunks written in one call, rows kept for the expansion too, padded batch
        dict(name="lwrite prefill 16384", op="lwrite", tokens=16384, seqs=41, heads=16, bs=32, dtype="bf16",
             interleaved=False, norm=True, padded=13, copy=True),
        # four short chats, 16 heads: the smallest decode step
        dict(name="latent tiny", op="latent", seqs=4, lo=1, hi=100, n_lo=1, n_hi=1, heads=16, bs=16, dtype="bf16",
             tree=False),
        # 64 chats of 512 to 4096 tokens, all 128 heads on one GPU
        dict(name="latent 64x4096 128h", op="latent", seqs=64, lo=512, hi=4096, n_lo=1, n_hi=1, heads=128, bs=16,
             dtype="bf16", tree=False),
        # eight documents of 131072 tokens, 16 heads, trees of up to four drafted tokens
        dict(name="latent 8x131072 16h 4", op="latent", seqs=8, lo=131072, hi=131072, n_lo=1, n_hi=4, heads=16, bs=32,
             dtype="fp16", tree=True),
        # a short prompt alone
        dict(name="prompt 100", op="prompt", seqs=1, lo=100, hi=100, prefix=0, heads=16, dtype="bf16"),
        # seven ragged prompts, one of them behind a cached prefix
        dict(name="prompt 7x1537", op="prompt", seqs=7, lo=1, hi=1537, prefix=513, heads=40, dtype="fp16"),
        # two long prompts, all 128 heads
        dict(name="prompt 2x8192 128h", op="prompt", seqs=2, lo=8192, hi=8192, prefix=0, heads=128, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "latent", "latent", "lwrite", "prompt", "prompt"])
    dtype = rng.choice(["bf16", "fp16"])
    bs = rng.choice([16, 32])
    if op == "lwrite":
        heads = rng.choice([1, 8, 16, 40, 64, 128])
        tokens = min(_log_int(rng, 1, 1500000 // (heads + 80)), 16384)
        seqs = tokens if rng.random() < 0.3 else _log_int(rng, 1, max(1, tokens // 8))
        return dict(op=op, tokens=tokens, seqs=seqs, heads=heads, bs=bs, dtype=dtype, interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.8, padded=rng.choice([0, 0, 1, 13]), copy=rng.random() < 0.5)
    if op == "prompt":
        heads = rng.choice([1, 8, 16, 40, 64, 128])
        seqs = _log_int(rng, 1, 16)
        hi = _log_int(rng, 1, min(8192, int(math.sqrt(8e9 / (heads * seqs)))))
        return dict(op=op, seqs=seqs, lo=rng.choice([1, max(1, hi // 4), hi]), hi=hi, prefix=rng.choice([0, 0, 1, 100, 1000]),
                    heads=heads, dtype=dtype)
    n_hi = rng.choice([1, 2, 4, 7, 16, 31, 64])
    n_lo = rng.choice([1, n_hi])
    seqs = _log_int(rng, 1, 128)
    if op == "tree":
        hq, hkv = rng.choice([(32, 8), (64, 8), (40, 40), (4, 1), (24, 3), (16, 1), (12, 2), (7, 7)])
        hi = _log_int(rng, n_hi, min(131072, max(2 * n_hi, 250000000 // (seqs * hq * max(n_hi, 8)))))
        return dict(op=op, seqs=seqs, lo=rng.choice([n_hi, max(n_hi, hi // 8), hi]), hi=hi, n_lo=n_lo, n_hi=n_hi, hq=hq,
                    hkv=hkv, bs=bs, dtype=dtype, tree=rng.random() < 0.7)
    heads = rng.choice([1, 8, 16, 40, 64, 128])
    hi = _log_int(rng, n_hi, min(131072, max(2 * n_hi, 30000000 // (seqs * max(heads * n_hi, 32)))))
    return dict(op=op, seqs=seqs, lo=rng.choice([n_hi, max(n_hi, hi // 8), hi]), hi=hi, n_lo=n_lo, n_hi=n_hi, heads=heads,
                bs=bs, dtype=dtype, tree=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _table():
    """cos and sin of every position, [MAX_POSITION, ROT]: cosines of the ROT / 2 angles, then sines."""
    inv = BASE ** (-torch.arange(0, ROT, 2, dtype=torch.float64, device="cuda") / ROT)
    a = torch.arange(MAX_POSITION, dtype=torch.float64, device="cuda")[:, None] * inv[None, :]
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _sizes(case, host):
    """The batch of a case: (context length, drafted tokens) of each sequence, or a prompt's (keys, new tokens).  The sizes
    are the case's own, so that every seed's outputs have one shape; their order is the seed's."""
    of = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    lens = [of.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    lens[of.randrange(len(lens))] = case["hi"]
    if case["op"] == "prompt":
        both = [(L, L) for L in lens]
        both[0] = (lens[0] + case["prefix"], lens[0])
    else:
        both = [(L, min(L, of.randint(case["n_lo"], case["n_hi"]))) for L in lens]
    host.shuffle(both)
    return [b[0] for b in both], [b[1] for b in both]


def _starts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _masks(host, counts):
    """A random tree over each sequence's drafted tokens: token i hangs below an earlier one, or below the context."""
    masks = []
    for n in counts:
        mine = []
        for i in range(n):
            parent = host.randint(-1 if host.random() < 0.1 else max(0, i - 4), i - 1) if i else -1
            m = (1 << i) | (mine[parent] if parent >= 0 else 0)
            mine.append(m)
        masks += mine
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device="cuda")


def _tables(g, lens, bs):
    """Scattered blocks of every sequence, [seqs, most blocks] (unused entries -1), and the pool's size."""
    n = [-(-L // bs) for L in lens]
    nb = sum(n) + sum(n) // 8 + 1
    perm = torch.randperm(nb, generator=g, device="cuda").int()
    width = max(1, max(n))
    nn = torch.tensor(n, device="cuda")
    j = torch.arange(width, device="cuda")[None, :] + (nn.cumsum(0) - nn)[:, None]
    inside = torch.arange(width, device="cuda")[None, :] < nn[:, None]
    return torch.where(inside, perm[j.clamp(max=nb - 1)], -1).int().contiguous(), nb


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cached_inputs(case, seed):
    host, g = random.Random(seed), _gen(seed)
    dt, bs = TYPES[case["dtype"]], case["bs"]
    lens, counts = _sizes(case, host)
    bt, nb = _tables(g, lens, bs)
    T = sum(counts)
    st = dict(case=case, block_tables=bt, context_lens=_ints(lens), query_starts=_ints(_starts(counts)), lens=lens,
              counts=counts, masks=_masks(host, counts) if case["tree"] else None)
    if case["op"] == "tree":
        hq, hkv = case["hq"], case["hkv"]
        gain = torch.exp(0.5 * _randn(g, hkv, 1, D))  # some key channels are larger, as in trained models
        st["q"] = _randn(g, T, hq, D).to(dt)
        st["k_cache"] = _randn(g, nb, hkv, bs, D).mul_(gain).to(dt)
        st["v_cache"] = _randn(g, nb, hkv, bs, D).to(dt)
        st["scale"] = D ** -0.5
    else:
        st["q"] = _randn(g, T, case["heads"], ROW).to(dt)
        st["cache"] = _randn(g, nb, bs, ROW).to(dt)
        st["scale"] = (D + ROT) ** -0.5
    return st


def _write_inputs(case, seed):
    """New rows of sequences that start at a position of their own; `padded` rows behind them have no slot."""
    host, g = random.Random(seed), _gen(seed)
    T, S, bs, H = case["tokens"], case["seqs"], case["bs"], case["heads"]
    if S == T:
        counts = [1] * T
    else:
        cuts = sorted(host.sample(range(1, T), S - 1)) if S > 1 else []
        counts = [b - a for a, b in zip([0] + cuts, cuts + [T])]
    firsts = [host.randrange(0, MAX_POSITION - n + 1) if host.random() < 0.8 else 0 for n in counts]
    cnt = torch.tensor(counts)
    pos = torch.repeat_interleave(torch.tensor(firsts) - (cnt.cumsum(0) - cnt), cnt) + torch.arange(T)
    blocks = [(p + n - 1) // bs - p // bs + 1 for p, n in zip(firsts, counts)]
    first = [a - p // bs for a, p in zip(_starts(blocks), firsts)]
    logical = (pos // bs + torch.repeat_interleave(torch.tensor(first), cnt)).cuda()
    pos = pos.cuda()
    nb = (T if S == T else T // bs + 2 * S) * 5 // 4 + 1
    perm = torch.randperm(nb, generator=g, device="cuda")
    pad = torch.full((case["padded"],), -1, dtype=torch.int64, device="cuda")
    rows, dt = T + case["padded"], TYPES[case["dtype"]]
    return dict(case=case, q=_randn(g, rows, H, D + ROT).to(dt),       # as the query projection leaves it
                kv=(_randn(g, rows, ROW) * 3.0).to(dt),                 # and the latent's
                positions=torch.cat([pos, torch.zeros_like(pad)]), slots=torch.cat([perm[logical] * bs + pos % bs, pad]),
                cos_sin=_table(), kv_norm=(1.0 + 0.1 * _randn(g, LATENT)).to(dt) if case["norm"] else None,
                cache=_randn(g, nb, bs, ROW).to(dt), q_out=torch.zeros(rows, H, ROW, dtype=dt, device="cuda"),
                kv_out=torch.zeros(rows, ROW, dtype=dt, device="cuda") if case["copy"] else None)


def _prompt_inputs(case, seed):
    host, g = random.Random(seed), _gen(seed)
    dt, H = TYPES[case["dtype"]], case["heads"]
    keys, new = _sizes(case, host)
    Tq, Tk = sum(new), sum(keys)
    rows = _randn(g, Tk, ROW).to(dt)   # the prompts' latent rows; the heads share the last 64 values
    return dict(case=case, q=_randn(g, Tq, H, D + ROT).to(dt), kv=_randn(g, Tk, H, 2 * D).to(dt), k_rope=rows[:, LATENT:],
                query_starts=_ints(_starts(new)), key_starts=_ints(_starts(keys)), new=new, keys=keys, longest=max(new),
                scale=(D + ROT) ** -0.5)


def prepare(case, seed):
    if case["op"] == "lwrite":
        return _write_inputs(case, seed)
    if case["op"] == "prompt":
        return _prompt_inputs(case, seed)
    return _cached_inputs(case, seed)


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return {"tree": _own_tree, "lwrite": _own_write, "latent": _own_latent, "prompt": _own_prompt}[op](st)
    return {"tree": _tree, "lwrite": _write, "latent": _latent, "prompt": _prompt}[op](st)


def _own_tree(st):
    import paged_kv_cache_11_gb300 as pkv
    return pkv.paged_attention_tree(st["q"], st["k_cache"], st["v_cache"], st["block_tables"], st["context_lens"],
                                    st["query_starts"], st["masks"], st["scale"])


def _own_write(st):
    import paged_kv_cache_11_gb300 as pkv
    pkv.paged_latent_append_rope(st["q"][:, :, D:], st["kv"], st["positions"], st["cos_sin"], st["slots"], st["cache"],
                                 kv_norm=st["kv_norm"], norm_eps=EPS, interleaved=st["case"]["interleaved"],
                                 q_out=st["q_out"][:, :, LATENT:], kv_out=st["kv_out"])
    return dict(q=st["q_out"], cache=st["cache"], kv=st["kv_out"])


def _own_latent(st):
    import paged_kv_cache_11_gb300 as pkv
    return pkv.paged_latent_decode(st["q"], st["cache"], st["block_tables"], st["context_lens"], st["scale"],
                                   query_starts=st["query_starts"], tree_masks=st["masks"])


def _own_prompt(st):
    import paged_kv_cache_11_gb300 as pkv
    return pkv.latent_attention_prefill(st["q"], st["kv"], st["k_rope"], st["query_starts"], st["key_starts"], st["scale"],
                                        max_query_len=st["longest"])


# the plain forms
def _visible(n, L, masks, device):
    """[n, L]: does drafted token i attend position t?"""
    i = torch.arange(n, device=device)
    if masks is None:
        own_part = i[None, :] <= i[:, None]
    else:
        own_part = (masks[:, None] >> i[None, :]) & 1 == 1
    return torch.cat([torch.ones(n, L - n, dtype=torch.bool, device=device), own_part], dim=1)


def _weights(s, seen):
    """Softmax over the last axis of the places seen, in 32 bits; rows that see nothing are zeros."""
    s = torch.where(seen, s, -math.inf)
    m = s.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s - m)
    total = p.sum(dim=-1, keepdim=True)
    return torch.where(total > 0, p / total, 0.0)


def _each(st):
    """First drafted row, drafted tokens, context length, block ids and masks of each sequence."""
    a, bs = 0, st["case"]["bs"]
    for s, (n, L) in enumerate(zip(st["counts"], st["lens"])):
        masks = None if st["masks"] is None else st["masks"][a:a + n]
        yield a, n, L, st["block_tables"][s, : -(-L // bs)].long(), masks
        a += n


def _tree(st):
    q = st["q"]
    hq, hkv = q.shape[1], st["k_cache"].shape[1]
    out = torch.empty_like(q)
    for a, n, L, ids, masks in _each(st):
        k, v = (st[c][ids].float().transpose(0, 1).reshape(hkv, -1, D)[:, :L] for c in ("k_cache", "v_cache"))
        x = q[a:a + n].float().view(n, hkv, hq // hkv, D).permute(1, 2, 0, 3)      # [hkv, group, n, D]
        s = torch.matmul(x.reshape(hkv, -1, D), k.transpose(1, 2)).view(hkv, hq // hkv, n, L) * st["scale"]
        p = _weights(s, _visible(n, L, masks, q.device))
        o = torch.matmul(p.view(hkv, -1, L), v).view(hkv, hq // hkv, n, D)
        out[a:a + n] = o.permute(2, 0, 1, 3).reshape(n, hq, D).to(q.dtype)
    return out


def _latent(st):
    q = st["q"]
    H = q.shape[1]
    out = q.new_empty(q.shape[0], H, LATENT)
    for a, n, L, ids, masks in _each(st):
        rows = st["cache"][ids].float().reshape(-1, ROW)[:L]
        s = torch.matmul(q[a:a + n].float().transpose(0, 1).reshape(-1, ROW), rows.t()).view(H, n, L) * st["scale"]
        p = _weights(s, _visible(n, L, masks, q.device))
        o = torch.matmul(p.view(-1, L), rows[:, :LATENT]).view(H, n, LATENT)
        out[a:a + n] = o.transpose(0, 1).to(q.dtype)
    return out


def _turned(x, row, interleaved):
    """x [..., ROT] turned by the angles whose cosines and sines are row [..., ROT]."""
    c, s = row[..., : ROT // 2], row[..., ROT // 2:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    a, b = x[..., : ROT // 2], x[..., ROT // 2:]
    return torch.cat([a * c - b * s, b * c + a * s], dim=-1)


def _write(st):
    n, bs, inter = st["case"]["tokens"], st["case"]["bs"], st["case"]["interleaved"]
    row = st["cos_sin"][st["positions"][:n]]
    c, dt = st["kv"][:n, :LATENT].float(), st["kv"].dtype
    if st["kv_norm"] is not None:
        c = c / torch.sqrt((c * c).mean(dim=-1, keepdim=True) + EPS) * st["kv_norm"].float()
    new = torch.cat([c, _turned(st["kv"][:n, LATENT:].float(), row, inter)], dim=-1).to(dt)
    slots = st["slots"][:n]
    st["cache"][slots // bs, slots % bs] = new
    st["q_out"][:n, :, LATENT:] = _turned(st["q"][:n, :, D:].float(), row[:, None, :], inter).to(dt)
    if st["kv_out"] is not None:
        st["kv_out"][:n] = new
    return dict(q=st["q_out"], cache=st["cache"], kv=st["kv_out"])


def _prompt(st):
    q = st["q"]
    H = q.shape[1]
    out = q.new_empty(q.shape[0], H, D)
    a = b = 0
    for n, L in zip(st["new"], st["keys"]):
        kv, shared = st["kv"][b:b + L], st["k_rope"][b:b + L].float()
        seen = torch.arange(L, device=q.device)[None, :] <= torch.arange(n, device=q.device)[:, None] + (L - n)
        step = max(1, (1 << 31) // (n * L))   # heads at a time: scores of 8 GB at most
        for h in range(0, H, step):
            x = q[a:a + n, h:h + step].float().transpose(0, 1)
            k, v = (kv[:, h:h + step, i:i + D].float().transpose(0, 1) for i in (0, D))
            s = torch.matmul(x[..., :D], k.transpose(1, 2)) + torch.matmul(x[..., D:], shared.t())
            out[a:a + n, h:h + step] = torch.matmul(_weights(s * st["scale"], seen), v).transpose(0, 1).to(q.dtype)
        a, b = a + n, b + L
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "lwrite":
        T, H = case["tokens"], case["heads"]
        return dict(bytes=T * (ROW * 2 * (3 if case["copy"] else 2) + 2 * H * ROT * 2 + 4 * ROT + 16),
                    flops=T * ((H + 1) * 3 * ROT + (4 * LATENT if case["norm"] else 0)))
    if op == "prompt":
        S, H = case["seqs"], case["heads"]
        n = (case["hi"] + (S - 1) * (case["lo"] + case["hi"]) / 2) / S
        n2 = (case["hi"] ** 2 + (S - 1) * (case["lo"] ** 2 + case["lo"] * case["hi"] + case["hi"] ** 2) / 3) / S
        pairs = S * (n2 + n) / 2 + n * case["prefix"]
        Tq, Tk = S * n, S * n + case["prefix"]
        return dict(bytes=2 * (Tq * H * (2 * D + ROT) + Tk * (H * 2 * D + ROT)), flops=2 * pairs * H * (2 * D + ROT))
    S = case["seqs"]
    tokens = case["hi"] + (S - 1) * (case["lo"] + case["hi"]) / 2
    n = (case["n_lo"] + case["n_hi"]) / 2
    if op == "tree":
        hq, hkv = case["hq"], case["hkv"]
        return dict(bytes=tokens * (hkv * 2 * D * 2 + 4 / case["bs"]) + S * n * (2 * hq * D * 2 + 8),
                    flops=4 * tokens * n * hq * D)
    H = case["heads"]
    return dict(bytes=tokens * (ROW * 2 + 4 / case["bs"]) + S * n * (H * (ROW + LATENT) * 2 + 8),
                flops=2 * tokens * n * H * (ROW + LATENT))


# ------------------------------------------------------------------ from the definitions, in 64 bits
MOST64 = 4e12   # operations in 64 bits that a card does in some seconds


def exact(case, seed):
    if case["op"] != "lwrite" and work(case)["flops"] > MOST64:
        return None
    st = prepare(case, seed)
    if case["op"] == "lwrite":
        return _written_exact(st)
    return _prompt_exact(st) if case["op"] == "prompt" else _attended_exact(st)


def _written_exact(st):
    n, bs = st["case"]["tokens"], st["case"]["bs"]
    x = st["kv"][:n].double()
    c = x[:, :LATENT]
    if st["kv_norm"] is not None:
        c = c * (c.pow(2).sum(-1, keepdim=True) / LATENT + EPS).rsqrt() * st["kv_norm"].double()
    t = st["cos_sin"][st["positions"][:n]].double()
    turn = torch.complex(t[:, : ROT // 2], t[:, ROT // 2:])

    def turned(y, by):
        if st["case"]["interleaved"]:
            z = torch.view_as_complex(y.reshape(*y.shape[:-1], ROT // 2, 2).contiguous()) * by
            return torch.view_as_real(z).reshape(y.shape)
        z = torch.complex(y[..., : ROT // 2].contiguous(), y[..., ROT // 2:].contiguous()) * by
        return torch.cat([z.real, z.imag], dim=-1)

    new = torch.cat([c, turned(x[:, LATENT:], turn)], dim=-1)
    cache, q = st["cache"].double(), st["q_out"].double()
    cache.view(-1, ROW).index_copy_(0, st["slots"][:n], new)
    q[:n, :, LATENT:] = turned(st["q"][:n, :, D:].double(), turn[:, None, :])
    kv = None
    if st["kv_out"] is not None:
        kv = st["kv_out"].double()
        kv[:n] = new
    return dict(q=q, cache=cache, kv=kv)


def _attended_exact(st):
    """Token by token: the positions that it attends are picked out first, then an ordinary softmax over them."""
    q, tree = st["q"].double(), st["case"]["op"] == "tree"
    out = torch.zeros(*q.shape[:2], D if tree else LATENT, dtype=torch.float64, device="cuda")
    tables, bs, row = st["block_tables"].long(), st["case"]["bs"], 0
    for s, (n, L) in enumerate(zip(st["counts"], st["lens"])):
        t = torch.arange(L, device="cuda")
        blk, off = tables[s, t // bs], t % bs
        if tree:
            k, v = st["k_cache"][blk, :, off].double(), st["v_cache"][blk, :, off].double()   # [L, hkv, D]
            group = q.shape[1] // k.shape[1]
        else:
            k = st["cache"][blk, off].double()
        for i in range(n):
            m = -1 if st["masks"] is None else int(st["masks"][row])
            keep = L - n + torch.tensor([j for j in range(n) if (m >> j & 1 if st["masks"] is not None else j <= i)],
                                        dtype=torch.int64, device="cuda")
            at = torch.cat([t[: L - n], keep])
            if at.numel():
                if tree:
                    z = torch.einsum("hgd,thd->hgt", q[row].view(-1, group, D), k[at]) * st["scale"]
                    out[row] = torch.einsum("hgt,thd->hgd", torch.softmax(z, -1), v[at]).reshape(-1, D)
                else:
                    out[row] = torch.softmax(q[row] @ k[at].t() * st["scale"], -1) @ k[at][:, :LATENT]
            row += 1
    return out


def _prompt_exact(st):
    q = st["q"].double()
    out = torch.zeros(*q.shape[:2], D, dtype=torch.float64, device="cuda")
    qs, ks = st["query_starts"].tolist(), st["key_starts"].tolist()
    for s in range(len(qs) - 1):
        n, L = qs[s + 1] - qs[s], ks[s + 1] - ks[s]
        kv = st["kv"][ks[s]:ks[s + 1]].double()
        shared = st["k_rope"][ks[s]:ks[s + 1]].double()
        for a in range(0, n, 256):          # a strip of queries at a time, over the keys that its last one sees
            b = min(n, a + 256)
            seen = L - n + b
            key = torch.cat([kv[:seen, :, :D], shared[:seen, None].expand(-1, q.shape[1], -1)], dim=-1)
            z = torch.einsum("qhd,khd->hqk", q[qs[s] + a:qs[s] + b], key) * st["scale"]
            hide = torch.ones(b - a, seen, dtype=torch.bool, device="cuda").triu(L - n + a + 1)
            z.masked_fill_(hide, -math.inf)
            out[qs[s] + a:qs[s] + b] = torch.einsum("hqk,khd->qhd", torch.softmax(z, -1), kv[:seen, :, D:])
    return out
