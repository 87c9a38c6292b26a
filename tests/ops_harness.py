"""References in 64 bits, on the CPU, of the operators beside the MoE layer,
and makers of their inputs.

Formats: a code is an e4m3fn byte, a scale byte b means 2^(b-127).  A page and
kv head holds K of token t, dimension d at byte ((d / 16) * 64 + t) * 16 +
d % 16 and V at ((t % 16 / 4) * D + d) * 16 + t / 16 * 4 + t % 4.
"""

from __future__ import annotations

import math

import torch

PAGE, BLOCK = 64, 128


def _table():
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 512 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        x = math.nan if c & 127 == 127 else x
        v.append(-x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64)


VALUE = _table()
CODES_UP = torch.tensor([c for c in range(127)], dtype=torch.int64)  # ascending values


def encode(x):
    """Codes of float64 values: nearest, ties to the even code; NaN and
    infinities are the code 0x7f (either sign counts as NaN)."""
    vals = VALUE[:127]
    a = x.abs()
    hi = torch.searchsorted(vals, a.nan_to_num(0, 0, 0).contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - vals[lo], vals[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    c = torch.where(up, hi, lo)
    c = torch.where(a >= 448, torch.full_like(c, 126), c)
    c = c + 128 * (torch.signbit(x)).long()
    return torch.where(torch.isfinite(x), c, torch.full_like(c, 127)).to(torch.uint8)


def same_codes(a, b):
    """Equal bytes; every NaN code is the same."""
    a, b = a.long(), b.long()
    return torch.where(a % 128 == 127, 127, a).equal(torch.where(b % 128 == 127, 127, b))


def power(e):
    return torch.tensor([math.ldexp(1.0, k) for k in range(-400, 401)], dtype=torch.float64)[e.long() + 400]


def scale_exp(amax):
    e = torch.full(amax.shape, -127, dtype=torch.int64)
    for k in range(-127, 128):
        e = torch.where(amax > 448 * math.ldexp(1.0, k), k + 1, e)
    return e


def finite_amax(x, dims):
    return torch.where(torch.isfinite(x), x.abs(), 0.0).amax(dims)


def quant_ref(x, limit=None):
    """(codes, scale bytes) of x [M, K] (or [M, 2K] with limit)."""
    x = x.double().cpu()
    if limit is not None:
        K = x.shape[1] // 2
        g, u = x[:, :K].clamp(max=limit), x[:, K:].clamp(-limit, limit)
        x = g / (1 + torch.exp(-g)) * u
    M, K = x.shape
    x = x.view(M, K // BLOCK, BLOCK)
    e = scale_exp(finite_amax(x, 2))
    return encode(x * power(-e)[..., None]).view(M, K), (e + 127).to(torch.uint8)


def dequant_rows(codes, scales):
    return VALUE[codes.long()] * power(scales.long() - 127).repeat_interleave(BLOCK, 1)


def dequant_w(w, w_scale):
    N, K = w.shape
    s = power(w_scale.long() - 127) if w_scale.dtype == torch.uint8 else w_scale.double()
    return VALUE[w.long()] * s.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)


def rand_codes(g, shape):
    """Codes of every finite value, both signs."""
    c = torch.randint(0, 254, shape, generator=g)
    return torch.where(c >= 127, c + 1, c).to(torch.uint8)


def normal_codes(g, shape, std=64.0):
    return encode((torch.randn(shape, generator=g, dtype=torch.float64) * std).clamp(-448, 448))


def at_k(D):
    t, d = torch.arange(PAGE)[:, None], torch.arange(D)[None]
    return (d // 16 * PAGE + t) * 16 + d % 16  # [64, D]


def at_v(D):
    t, d = torch.arange(PAGE)[:, None], torch.arange(D)[None]
    return (t % 16 // 4 * D + d) * 16 + t // 16 * 4 + t % 4


class CacheCase:
    """A cache on the CPU: lens (new tokens included), new tokens per sequence
    qs, extra rows behind the last sequence, its pool with every byte random
    (NaN codes too) behind the sequences' last tokens."""

    def __init__(self, seed, lens, qs, heads, kv, D, max_pages=None, extra=2, spare=3, max_q=None):
        g = torch.Generator().manual_seed(seed)
        self.g, self.lens, self.qs = g, list(lens), list(qs)
        self.heads, self.kv, self.D = heads, kv, D
        self.B = len(self.lens)
        need = [-(-n // PAGE) for n in self.lens]
        self.P = max_pages or max(need + [1])
        self.max_q = max_q or max(self.qs + [1])
        self.pages = sum(need) + spare
        perm = torch.randperm(self.pages, generator=g)
        self.table = torch.full((self.B, self.P), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n].int()
            at += n
        self.start = [0]
        for q in self.qs:
            self.start.append(self.start[-1] + q)
        self.T = self.start[-1] + extra
        self.pool = normal_codes(g, (self.pages, 2, kv, PAGE * D), 90.0)
        self.scale = torch.randint(118, 122, (self.pages, 2, kv), generator=g).to(torch.uint8)
        for b, n in enumerate(self.lens):
            if n % PAGE:  # stale bytes behind the last token
                p = int(self.table[b, n // PAGE])
                for s, at_ in ((0, at_k(D)), (1, at_v(D))):
                    idx = at_[n % PAGE:].reshape(-1)
                    self.pool[p, s][:, idx] = torch.randint(0, 256, (kv, idx.numel()), generator=g).to(torch.uint8)

    def rows(self, heads, scale=1.0):
        x = torch.randn(self.T, heads, self.D, generator=self.g) * scale
        return x.to(torch.bfloat16)

    def dev(self, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        return dict(pool=self.pool.to(device), pool_scale=self.scale.to(device),
                    page_table=self.table.to(device), seq_lens=torch.tensor(self.lens, **i32),
                    q_start=torch.tensor(self.start, **i32))

    def kv_of(self, b, h, pool=None, scale=None):
        """K and V [len, D] in float64 of sequence b, kv head h."""
        pool = self.pool if pool is None else pool
        scale = self.scale if scale is None else scale
        n = self.lens[b]
        ids = self.table[b, :-(-n // PAGE)].long()
        e = power(scale[ids].long() - 127)
        k = VALUE[pool[ids, 0, h][:, at_k(self.D)].long()] * e[:, 0, h, None, None]
        v = VALUE[pool[ids, 1, h][:, at_v(self.D)].long()] * e[:, 1, h, None, None]
        return k.flatten(0, 1)[:n], v.flatten(0, 1)[:n]


def attend_ref(case, q, sm_scale):
    """out [T, heads, D] (NaN rows where no sequence), mass [B, P] and the
    bounds of both for the kernel's arithmetic:

    A score sums D exact products in fp32: off by at most (D + 4) 2^-23 sum|q k|
    sm_scale log2(e) in base 2 with its two scalings; 2^x is off by about
    2^-22 more with the rounding of its argument (|x| 2^-24 ln 2).  So every
    probability is off by 2 (ln2 es + 2^-22 + ...) of itself, numerator and
    denominator.  As f16 it is off by 2^-11 of itself or 2^-25; the sums over n
    tokens add (64 + pages) 2^-23 of the sum of |p v|; the output's rounding
    is 2^-8 of it.
    """
    out = torch.full((case.T, case.heads, case.D), math.nan, dtype=torch.float64)
    tol = torch.zeros_like(out)
    mass = torch.zeros(case.B, case.P, dtype=torch.float64)
    mtol = torch.zeros_like(mass)
    G = case.heads // case.kv
    for b in range(case.B):
        n, nq = case.lens[b], case.qs[b]
        if not nq:
            continue
        np_ = -(-n // PAGE)
        seen = torch.arange(n)[None] < n - nq + 1 + torch.arange(nq)[:, None]
        for h in range(case.kv):
            k, v = case.kv_of(b, h)
            for a in range(h * G, (h + 1) * G):
                qa = q[case.start[b]:case.start[b + 1], a].double()
                s = (qa @ k.t() * sm_scale).masked_fill(~seen, -math.inf)
                p = torch.softmax(s, 1)
                vz = torch.where(torch.isnan(v), 0.0, v)
                o = p @ vz
                nan = (seen.double() @ torch.isnan(v).double()) > 0
                es = (case.D + 4) * 2.0 ** -23 * (qa.abs() @ k.abs().t()).masked_fill(~seen, 0).amax(1) * abs(sm_scale)
                top = s.masked_fill(~seen, 0).abs().amax(1) * 1.4427
                ep = 2 * (es + 2.0 ** -21 + top * 2.0 ** -23) + (64 + np_) * 2.0 ** -23
                pa, va = p @ vz.abs(), vz.abs().sum(0)
                out[case.start[b]:case.start[b + 1], a] = torch.where(nan, math.nan, o)
                l = torch.exp(s - s.amax(1, keepdim=True)).sum(1)
                tol[case.start[b]:case.start[b + 1], a] = (
                    (ep + 2.0 ** -11)[:, None] * pa + 2.0 ** -25 * va[None] / l[:, None]
                    + 2.0 ** -8 * o.abs())
                pm = torch.nn.functional.pad(p.nan_to_num(0), (0, np_ * PAGE - n)).view(nq, np_, PAGE).sum(2)
                mass[b, :np_] += pm.sum(0)
                # the record is log2 of the page's share: rounded at its size
                mtol[b, :np_] += (pm * (ep + (top + 30) * 2.0 ** -22)[:, None]).sum(0)
        # and a page's share of a row below fp32's least normal number is 0
        mtol[b] += mass[b] * (case.heads * nq + 4) * 2.0 ** -23 + case.heads * nq * 2.0 ** -125
    return out, tol, mass, mtol


def append_ref(case, k, v):
    """(pool, scale) after the append."""
    pool, scale = case.pool.clone(), case.scale.clone()
    for b in range(case.B):
        n, q = case.lens[b], case.qs[b]
        past = n - q
        for pi in range(past // PAGE, -(-n // PAGE) if q else 0):
            page = int(case.table[b, pi])
            if not 0 <= page < case.pages:
                continue
            lo, hi = max(past, pi * PAGE) - pi * PAGE, min(n, pi * PAGE + PAGE) - pi * PAGE
            r0 = case.start[b] + pi * PAGE - past
            for s, x, at in ((0, k, at_k(case.D)), (1, v, at_v(case.D))):
                for h in range(case.kv):
                    new = x[r0 + lo:r0 + hi, h].double()
                    e = int(scale_exp(finite_amax(new, (0, 1))))
                    was = int(scale[page, s, h]) - 127
                    if lo:
                        e = max(e, was)
                        old = at[:lo].reshape(-1)
                        if e > was:
                            vals = VALUE[pool[page, s, h, old].long()] * math.ldexp(1.0, was - e)
                            pool[page, s, h, old] = encode(vals)
                    pool[page, s, h, at[lo:hi].reshape(-1)] = encode(new * math.ldexp(1.0, -e)).reshape(-1)
                    scale[page, s, h] = e + 127
    return pool, scale


def evict_ref(table, lens, mass, keep, sink, recent):
    B, P = table.shape
    out = dict(out_table=torch.full((B, P), -1, dtype=torch.int32), out_lens=torch.zeros(B, dtype=torch.int32),
               out_mass=torch.zeros(B, P), freed=torch.full((B, P), -1, dtype=torch.int32),
               n_freed=torch.zeros(B, dtype=torch.int32))
    for b in range(B):
        fits = 0 <= lens[b] <= PAGE * P
        n = -(-int(lens[b]) // PAGE) if fits else P
        key = [math.inf if math.isnan(m) else m for m in mass[b].tolist()]
        nan = [math.isnan(m) for m in mass[b].tolist()]
        rivals = [i for i in range(n) if sink <= i < n - recent] if fits else []
        drop = sorted(rivals, key=lambda i: (nan[i], key[i], -i))[:max(0, n - keep) if fits else 0]
        left, gone = [i for i in range(n) if i not in set(drop)], sorted(drop)
        out["out_table"][b, :len(left)] = table[b, left]
        out["out_mass"][b, :len(left)] = mass[b, left]
        out["freed"][b, :len(gone)] = table[b, gone]
        out["n_freed"][b], out["out_lens"][b] = len(gone), int(lens[b]) - PAGE * len(gone)
    return out
