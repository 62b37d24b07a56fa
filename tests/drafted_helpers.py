"""Plain 64-bit forms of the attention calls on drafted tokens, latent caches and prompts, and the inputs of their tests.

Error bounds used by the tests, for an output y = sum_t w_t v_t of the softmax weights w, with A = sum_t w_t |v_t| and u half a
step of the 16-bit type (2^-8 bf16, 2^-11 fp16):
* a weight before it is normalised is rounded once, by a factor 1 + d, |d| <= u, and divided by the sum of the rounded ones, so
  y moves by at most sum_t w_t |d_t| |v_t - y| / (1 - u) <= 1.01 u (A + |y|); the output's rounding adds u |y|.
* weights below fp16's normal range (2^-14 of the largest, which is 1 at least) are off by 2^-25 at most: 2^-25 n max |v|
  for n tokens (bf16 has fp32's range).
* a score is summed in fp32, 16 products at a time: K / 16 + 4 additions of 2^-22 of sum |q k| each, e in all; and the weight's
  exponential and its argument are good to 2^-16 for scores up to 2^7: y moves by at most (2 e + 2^-15) A.
* every sum over n tokens in fp32: n / 16 + 4 additions of 2^-22 of A.
"""
import torch

D, LATENT, ROPE = 128, 512, 64
ROW = LATENT + ROPE
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
SENTINEL = -7.0  # of output rows that belong to no sequence


def attend64(q, k, v, seen, scale, dtype):
    """q [H, n, K], k [H, L, K], v [H, L, V] (64 bits; heads may be broadcast), seen [n, L] -> (out [H, n, V], bound of each
    value).  Tokens that no weight falls on count nothing, whatever they hold."""
    zero = torch.zeros((), dtype=torch.float64, device=q.device)
    keep = seen.any(0)
    k = torch.where(keep[:, None], k, zero)
    v = torch.where(keep[:, None], v, zero)
    s = torch.where(seen, q @ k.transpose(-1, -2) * scale, -torch.inf)
    m = s.amax(-1, keepdim=True) if s.shape[-1] else zero
    p = torch.exp(s - torch.where(torch.isinf(m) & (m < 0), zero, m))
    total = p.sum(-1, keepdim=True)
    w = torch.where(total > 0, p / torch.where(total > 0, total, zero + 1), torch.where(torch.isnan(total), total, zero))
    y, a = w @ v, w @ v.abs()
    u = U[dtype]
    n = seen.shape[1]
    mag = (q.abs() @ k.abs().transpose(-1, -2) * abs(scale) * seen).amax(-1, keepdim=True) if n else zero
    e = (q.shape[-1] / 16 + 4) * 2.0 ** -22 * mag
    bound = 1.01 * u * (a + y.abs()) + u * y.abs() + (2 * e + 2.0 ** -15 + (n / 16 + 4) * 2.0 ** -22) * a + 1e-30
    if dtype == torch.float16:
        bound = bound + 2.0 ** -25 * n * (v.abs().amax() if n else zero) + 2.0 ** -25
    return y, bound


def tree_masks(gen, counts, density=0.3):
    """Random trees: a token hangs below an earlier one or below the context."""
    out = []
    for n in counts:
        mine = []
        for i in range(n):
            parent = int(torch.randint(-1, i, (1,), generator=gen)) if i else -1
            mine.append((1 << i) | (mine[parent] if parent >= 0 else 0))
        out += mine
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in out], dtype=torch.int64)


class Batch:
    """Sequences of (context length, drafted tokens) over a scattered pool whose every place that no sequence holds is NaN.

    kind "tree": K and V pools; "latent": one pool of rows.  masks: "chain" (none), "tree", "random" (any bits).
    ``extra`` rows of q and out behind the last sequence belong to none."""

    def __init__(self, seed, seqs, heads, hkv=1, bs=16, dtype=torch.bfloat16, kind="tree", masks="tree", starts=True, extra=0,
                 scale=None, width=0, spare=3, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.dtype, self.bs, self.hkv, self.heads, self.device = kind, dtype, bs, hkv, heads, device
        self.lens, self.counts = [s[0] for s in seqs], [s[1] for s in seqs]
        row, val = (D, D) if kind == "tree" else (ROW, LATENT)
        self.val = val
        self.scale = (row ** -0.5 if kind == "tree" else 192 ** -0.5) if scale is None else scale
        nblk = [-(-L // bs) for L in self.lens]
        nb = sum(nblk) + spare
        perm = torch.randperm(nb, generator=g).int()
        w = max(1, width, *nblk) if nblk else 1
        self.tables = torch.full((len(seqs), w), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(nblk):
            self.tables[s, :n] = perm[at:at + n]
            at += n
        T = sum(self.counts) + extra
        gd = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *sh: torch.randn(*sh, generator=gd, device=device)
        self.q = rnd(T, heads, row).to(dtype)
        shape = (nb, hkv, bs, D) if kind == "tree" else (nb, bs, ROW)
        pools = [rnd(*shape).to(dtype) for _ in range(2 if kind == "tree" else 1)]
        used = torch.zeros(nb, bs, dtype=torch.bool)
        for s, L in enumerate(self.lens):
            t = torch.arange(L)
            used[self.tables[s, t // bs].long(), t % bs] = True
        used = used.to(device)
        for x in pools:
            x.masked_fill_(~(used[:, None, :, None] if kind == "tree" else used[:, :, None]), float("nan"))
        self.pools = pools
        self.tables = self.tables.to(device)
        self.context_lens = torch.tensor(self.lens, dtype=torch.int32, device=device)
        s = [0]
        for n in self.counts:
            s.append(s[-1] + n)
        self.starts_list = s
        self.starts = torch.tensor(s, dtype=torch.int32, device=device) if starts else None
        if masks == "chain":
            self.masks = None
        else:
            m = tree_masks(g, self.counts) if masks == "tree" else torch.randint(-2 ** 62, 2 ** 62, (sum(self.counts),), generator=g)
            self.masks = torch.cat([m, torch.full((extra,), -1)]).to(device)
        self.out = torch.full((T, heads, val), SENTINEL, dtype=dtype, device=device)

    def call(self, **kw):
        import paged_kv_cache_11_gb300 as pkv
        kw = {"out": self.out, **kw}
        if self.kind == "tree":
            return pkv.paged_attention_tree(self.q, *self.pools, self.tables, self.context_lens, self.starts, self.masks,
                                            self.scale, **kw)
        return pkv.paged_latent_decode(self.q, *self.pools, self.tables, self.context_lens, self.scale,
                                       query_starts=self.starts, tree_masks=self.masks, **kw)

    def seen(self, s):
        n, L = self.counts[s], self.lens[s]
        i = torch.arange(n, device=self.device)
        if self.masks is None:
            own = i[None, :] <= i[:, None]
        else:
            m = self.masks[self.starts_list[s]:self.starts_list[s] + n]
            own = (m[:, None] >> i[None, :]) & 1 == 1
        return torch.cat([torch.ones(n, max(0, L - n), dtype=torch.bool, device=self.device), own[:, :L]], dim=1)

    def rows(self, s):
        """Keys and values of sequence s in 64 bits, [heads, L, ...]."""
        t = torch.arange(self.lens[s], device=self.device)
        blk, off = self.tables[s, t // self.bs].long(), t % self.bs
        if self.kind == "tree":
            return [p[blk, :, off].double().transpose(0, 1).repeat_interleave(self.heads // self.hkv, 0) for p in self.pools]
        r = self.pools[0][blk, off].double()[None]
        return r, r[..., :LATENT]

    def expected(self, s):
        a, n = self.starts_list[s], self.counts[s]
        k, v = self.rows(s)
        y, b = attend64(self.q[a:a + n].double().transpose(0, 1), k, v, self.seen(s), self.scale, self.dtype)
        return y.transpose(0, 1), b.transpose(0, 1)

    def check(self, out=None, only=None, zeros=()):
        out = self.out if out is None else out
        for s in range(len(self.lens)) if only is None else only:
            a, n = self.starts_list[s], self.counts[s]
            got = out[a:a + n].double()
            if s in zeros or self.lens[s] == 0:
                assert (got == 0).all(), f"sequence {s}: not zeros"
                continue
            y, b = self.expected(s)
            off = (got - y).abs()
            assert (off <= b).all(), (f"sequence {s} (L {self.lens[s]}, n {n}): {int((~(off <= b)).sum())} of {off.numel()} off, "
                                      f"worst {float((off / b).nan_to_num(1e30).max()):.3g} of the bound")
        tail = out[self.starts_list[-1]:]
        assert (tail == SENTINEL).all(), "rows behind the last sequence were written"
