"""Plain 64-bit forms of the rotating cache writes and of the e4m3 cache, token
by token from their definitions, and the inputs of their tests.

Error bounds used by the tests (u: half a step of the output's type):
* a rotated (and normed) value is computed in fp32 from exact inputs: the norm
  is at most 16 roundings of 2^-24 (a 128-term sum in pairs, a root, a
  division, two products), the turn three more relative to |a| + |b| of its
  pair: together below 1.25 * 2^-20 (|a| + |b|), then one rounding u |y|.
* a stored e4m3 value is the nearest to y / scale: at most half a step from it,
  plus the fp32 error of y.
"""
import math

import numpy as np
import torch

D = 128
FP32_ERR = 1.25 * 2.0 ** -20
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half of the smallest step


def cos_sin_table(rows, rot, base=10000.0):
    if rot == 0:
        return None
    a = np.arange(rows)[:, None] * base ** (-np.arange(0, rot, 2) / rot)[None, :]
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32))


def turn(x, w, eps, row, interleaved):
    """One head row (float64 numpy [D]) -> (normed and rotated row, |a| + |b| of each value's pair)."""
    x = x.copy()
    if w is not None:
        x = x / math.sqrt(float((x * x).mean()) + eps) * w
    y, mag = x.copy(), np.abs(x)
    if row is not None:
        r = len(row) // 2
        for i in range(r):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
            c, s = float(row[i]), float(row[r + i])
            y[a], y[b] = x[a] * c - x[b] * s, x[b] * c + x[a] * s
            mag[a] = mag[b] = abs(x[a]) + abs(x[b])
    return y, mag


def to64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def p2_scale(a):
    """The smallest power of two >= a / 448, 2^-64 at least."""
    e = -64
    while a > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def e4m3_steps(r):
    """Step of e4m3 numbers at magnitude r."""
    r = np.abs(r)
    e = np.floor(np.log2(np.maximum(r, 2.0 ** -6)))
    return 2.0 ** (np.maximum(e, -6) - 3)


def e4m3_round(r):
    s = e4m3_steps(r)
    return np.round(r / s) * s  # numpy rounds halves to even


class Case:
    """Inputs of one append call on the CPU, and its expected results in 64 bits."""

    def __init__(self, seed, hq, hkv, bs, dtype, rot, interleaved, norm, slots, positions, num_blocks, max_position=512,
                 fused=True, fp8=False, eps=1e-5):
        g = torch.Generator().manual_seed(seed)
        n = len(slots)
        self.hq, self.hkv, self.bs, self.dtype, self.rot, self.inter, self.eps = hq, hkv, bs, dtype, rot, interleaved, eps
        rows = torch.randn(n, hq + 2 * hkv, D, generator=g).to(dtype)
        if fused:
            self.q, self.k, self.v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        else:
            self.q, self.k, self.v = (x.contiguous() for x in (rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]))
        self.fused, self.rows = fused, rows
        self.q_norm = (1 + 0.25 * torch.randn(D, generator=g)).to(dtype) if norm else None
        self.k_norm = (1 + 0.25 * torch.randn(D, generator=g)).to(dtype) if norm else None
        self.slots = torch.tensor(slots, dtype=torch.int64)
        self.positions = torch.tensor(positions, dtype=torch.int64) if rot else None
        self.cos_sin = cos_sin_table(max_position, rot)
        self.num_blocks, self.max_position, self.fp8 = num_blocks, max_position, fp8
        shape = (num_blocks, hkv, bs, D)
        if fp8:
            self.kc = (torch.randn(shape, generator=g) * 110).clamp(-448, 448).to(torch.float8_e4m3fn)
            self.vc = (torch.randn(shape, generator=g) * 110).clamp(-448, 448).to(torch.float8_e4m3fn)
            self.ks = torch.exp2(torch.randint(-9, -6, (num_blocks, hkv), generator=g).float())
            self.vs = torch.exp2(torch.randint(-9, -6, (num_blocks, hkv), generator=g).float())
        else:
            self.kc = torch.randn(shape, generator=g).to(dtype)
            self.vc = torch.randn(shape, generator=g).to(dtype)
            self.ks = self.vs = None
        self.q_out = torch.randn(n, hq, D, generator=g).to(dtype)

    def live(self):
        """Tokens that are written, and those whose query row becomes zeros."""
        ok, bad = [], []
        for t, s in enumerate(self.slots.tolist()):
            if s < 0:
                continue
            p = self.positions[t].item() if self.rot else 0
            fine = s < self.num_blocks * self.bs and (not self.rot or 0 <= p < self.max_position)
            (ok if fine else bad).append(t)
        return ok, bad

    def turned(self, which, t, h):
        x, w = (self.q, self.q_norm) if which == "q" else (self.k, self.k_norm)
        row = to64(self.cos_sin[self.positions[t]]) if self.rot else None
        return turn(to64(x[t, h]), to64(w), self.eps, row, self.inter)

    def to_dev(self, dev):
        """The call's tensors on the GPU (fused rows stay one tensor, sliced there)."""
        c = lambda t: None if t is None else t.to(dev)
        if self.fused:
            rows = self.rows.to(dev)
            q, k, v = rows[:, :self.hq], rows[:, self.hq:self.hq + self.hkv], rows[:, self.hq + self.hkv:]
        else:
            q, k, v = c(self.q), c(self.k), c(self.v)
        d = dict(q=q if self.hq else None, k=k, v=v, positions=c(self.positions), cos_sin=c(self.cos_sin),
                 slot_mapping=c(self.slots), k_cache=c(self.kc), v_cache=c(self.vc),
                 q_norm=c(self.q_norm) if self.hq else None, k_norm=c(self.k_norm), norm_eps=self.eps,
                 interleaved=self.inter, q_out=c(self.q_out) if self.hq else None)
        if self.fp8:
            d.update(k_scales=c(self.ks), v_scales=c(self.vs))
        return d

    def check_q(self, q_out):
        got, before = to64(q_out), to64(self.q_out)
        ok, bad = self.live()
        u, tiny = HALF[self.dtype], TINY[self.dtype]
        for t in range(len(self.slots)):
            for h in range(self.hq):
                if t in ok:
                    y, mag = self.turned("q", t, h)
                    assert (np.abs(got[t, h] - y) <= u * np.abs(y) + (1 + u) * FP32_ERR * mag + tiny).all(), (t, h)
                else:
                    assert np.array_equal(got[t, h], np.zeros(D) if t in bad else before[t, h]), (t, h)

    def check_pools16(self, kc, vc):
        k, v = to64(self.kc), self.vc.clone()
        tol = np.zeros_like(k)
        u, tiny = HALF[self.dtype], TINY[self.dtype]
        for t in self.live()[0]:
            b, o = divmod(self.slots[t].item(), self.bs)
            v[b, :, o] = self.v[t]
            for h in range(self.hkv):
                y, mag = self.turned("k", t, h)
                k[b, h, o] = y
                tol[b, h, o] = u * np.abs(y) + (1 + u) * FP32_ERR * mag + tiny
        assert (np.abs(to64(kc) - k) <= tol).all()   # rows that are not written: tolerance 0
        assert torch.equal(vc.cpu().view(torch.int16), v.view(torch.int16))

    def check_pools8(self, kc, vc, ks, vs):
        ok = self.live()[0]
        runs = {}
        for t in ok:
            runs.setdefault(self.slots[t].item() // self.bs, []).append(t)
        for which, cache0, scales0, cache, scales in (("k", self.kc, self.ks, kc, ks), ("v", self.vc, self.vs, vc, vs)):
            old_bytes, got_bytes = cache0.view(torch.uint8).numpy(), cache.cpu().view(torch.uint8).numpy()
            old_val, got_val = to64(cache0.float()), to64(cache.float())
            old_s, got_s = to64(scales0), to64(scales)
            for b in range(self.num_blocks):
                for h in range(self.hkv):
                    if b not in runs:
                        assert got_s[b, h] == old_s[b, h] or (np.isnan(got_s[b, h]) and np.isnan(old_s[b, h]))
                        assert np.array_equal(old_bytes[b, h], got_bytes[b, h])
                        continue
                    rows = {}
                    for t in runs[b]:
                        y, mag = self.turned("k", t, h) if which == "k" else (to64(self.v[t, h]), np.zeros(D))
                        rows[self.slots[t].item() % self.bs] = (y, mag)
                    first = min(rows)
                    a = max([np.abs(y[np.isfinite(y)]).max() for y, _ in rows.values() if np.isfinite(y).any()] or [0.0])
                    old = old_s[b, h]
                    usable = 2.0 ** -126 <= old < np.inf
                    # the choices below must not hang on the last bits of a
                    for edge in ([448 * old] if first and usable else []) + [448 * p2_scale(a), 224 * p2_scale(a)]:
                        exact = which == "v" or not (self.rot or self.k_norm is not None)
                        assert exact or a in (0, edge) or abs(a / edge - 1) > 2.0 ** -18  # (equal: a value that is not turned)
                    if first and usable and a <= 448 * old:
                        s = old
                    else:
                        s = p2_scale(a)
                    assert got_s[b, h] == s, (which, b, h, got_s[b, h], s)
                    for o in range(self.bs):
                        if o in rows:
                            y, mag = rows[o]
                            fine = np.isfinite(y)
                            assert np.isnan(got_val[b, h, o][~fine]).all()
                            r = y[fine] / s
                            off = np.abs(got_val[b, h, o][fine] - r)
                            if which == "v":
                                assert np.array_equal(got_val[b, h, o][fine], e4m3_round(r))
                            else:
                                step = np.maximum(e4m3_steps(r), e4m3_steps(got_val[b, h, o][fine]))
                                assert (off <= step / 2 + FP32_ERR * mag[fine] / s).all()
                        elif o < first and usable and s != old:
                            want = old_val[b, h, o]
                            nan = np.isnan(want)
                            assert np.array_equal(np.isnan(got_val[b, h, o]), nan)
                            assert np.array_equal(got_val[b, h, o][~nan], e4m3_round(want[~nan] * (old / s)))
                        else:
                            assert np.array_equal(old_bytes[b, h, o], got_bytes[b, h, o])


def runs_of_tokens(rng, spans, bs, num_blocks):
    """Slots and positions of sequences: `spans` lists (first position, tokens); blocks come shuffled from the pool."""
    perm = rng.permutation(num_blocks).tolist()
    slots, positions = [], []
    for p0, n in spans:
        blocks = {}
        for p in range(p0, p0 + n):
            b = blocks.setdefault(p // bs, perm[-1])
            if perm and b == perm[-1]:
                perm.pop()
            slots.append(b * bs + p % bs)
            positions.append(p)
    return slots, positions


def decode_inputs(seed, lens, hq, hkv, bs, dtype, wild_scales=False, poison=True):
    """An e4m3 pool, its scales, queries and tables; unread rows and scales are NaN when poisoned."""
    g = torch.Generator().manual_seed(seed)
    n = [-(-L // bs) for L in lens]
    nb = sum(n) + 3
    perm = torch.randperm(nb, generator=g).tolist()
    width = max(1, max(n, default=0))
    bt = torch.full((len(lens), width), -1, dtype=torch.int32)
    kc, vc = ((torch.randn(nb, hkv, bs, D, generator=g) * 110).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in range(2))
    if wild_scales:   # not powers of two, and far apart
        ks = torch.exp2(torch.randn(nb, hkv, generator=g) - 7)
        vs = torch.exp2(6 * torch.randn(nb, hkv, generator=g) - 7)
    else:
        ks, vs = (torch.exp2(torch.randint(-8, -5, (nb, hkv), generator=g).float()) for _ in range(2))
    used = torch.zeros(nb, bs, dtype=torch.bool)
    i = 0
    for s, L in enumerate(lens):
        for j in range(n[s]):
            bt[s, j] = perm[i]
            used[perm[i], : min(bs, L - j * bs)] = True
            i += 1
    if poison:
        for c in (kc, vc):
            raw = c.view(torch.uint8).transpose(1, 2)   # [nb, bs, hkv, D]
            raw[~used] = 0x7F
        for c in (ks, vs):
            c[~used.any(dim=1)] = math.nan
    q = torch.randn(len(lens), hq, D, generator=g).to(dtype)
    return dict(q=q, k_cache=kc, v_cache=vc, k_scales=ks, v_scales=vs, block_tables=bt,
                context_lens=torch.tensor(lens, dtype=torch.int32))


def decode_ref(inp, scale, out_dtype, heads=None):
    """Attention in 64 bits, and what the kernel's output may be off by, per value.

    A score is an fp32 sum of 128 exact products in 8 steps of 16, of a query
    whose row keeps 2^-25 of its largest value, times two fp32 factors: off by
    at most e_s = (8 + 3) 2^-23 S + 2^-25 qmax sum|k| with S = scale sum|q k|.
    A weight is off by 2 e_s relative (its own score and the sum's), by 2^-20
    for exp2 and the split of P, by the roundings of 2^-24 of the sums over one
    warp's units (L / 64 at most, an addition and a rescale each), of the
    products inside a unit and of the merges (fewer than 80), relative to the
    sum of weights times values, and by 2^-26 of the largest weight, or all of
    the weight where it is smaller, where fp16 has no smaller step (2^-24 in a P
    lifted by 2^7, of a scale of at least 2^-6 of O's unit).  The output's own
    rounding comes on top.
    """
    bs, hkv = inp["k_cache"].shape[2], inp["k_cache"].shape[1]
    B, hq, _ = inp["q"].shape
    out, tol = np.zeros((B, hq, D)), np.zeros((B, hq, D))
    q64 = to64(inp["q"])
    kraw, vraw = (inp[c].cpu().view(torch.uint8) for c in ("k_cache", "v_cache"))
    for s in range(B):
        L = int(inp["context_lens"][s])
        if L == 0:
            continue
        ids = inp["block_tables"][s, : -(-L // bs)].long().cpu()
        k, v = (to64(raw[ids].view(torch.float8_e4m3fn).float()) * to64(inp[f].cpu()[ids])[:, :, None, None]
                for raw, f in ((kraw, "k_scales"), (vraw, "v_scales")))
        k, v = (x.transpose(1, 0, 2, 3).reshape(hkv, -1, D)[:, :L] for x in (k, v))
        for h in range(hq) if heads is None else heads:
            kh, vh, qh = k[h * hkv // hq], v[h * hkv // hq], q64[s, h]
            z = scale * (kh @ qh)
            w = np.exp(z - z.max())
            l = w.sum()
            out[s, h] = (w @ vh) / l
            S = abs(scale) * (np.abs(kh) @ np.abs(qh)).max()
            e_s = 11 * 2.0 ** -23 * S + 2.0 ** -25 * abs(scale) * np.abs(qh).max() * np.abs(kh).sum(axis=1).max()
            spread = (w @ np.abs(vh)) / l
            tol[s, h] = ((2 * e_s + 2.0 ** -20 + (L / 32 + 80) * 2.0 ** -24) * spread +
                         np.minimum(w, 2.0 ** -26) @ np.abs(vh) / l)
    tol += HALF[out_dtype] * np.abs(out) + TINY[out_dtype]
    return out, tol
