"""The operators beside the MoE layer as cases to be timed and compared: the
block-scaled fp8 product with its activation quantiser, and the attention
over an 8-bit paged cache with its append and its eviction.

`run` computes a case in elementary torch operations, or with `own` set
through the package's entry points; `exact` computes it in 64 bits.

Formats
  codes   e4m3fn bytes; a scale byte b stands for 2^(b - 127)
  pool    [pages, 2, kv_heads, 64 * head_dim] codes: K of a page and head is
          [head_dim / 16][64 tokens][16], V is [4][head_dim][16] where byte
          4 a + c of piece g is token 16 a + 4 g + c
  scales  [pages, 2, kv_heads] bytes, one for K and one for V
"""

import math
import random

import torch

own = False

DEV = "cuda"
PAGE = 64
BLOCK = 128
F8 = torch.float8_e4m3fn
SINK, RECENT = 1, 2


def listed():
    return [
        # one decode token's activations, quantised for the next projection
        dict(name="quant_t1", op="quant", M=1, K=4096, limit=0.0),
        # a prompt chunk between the two products of a dense MLP
        dict(name="quant_swiglu_t4096", op="quant", M=4096, K=2048, limit=7.0),
        # the fused q, k, v projection of one decode token
        dict(name="product_t1", op="product", M=1, N=6144, K=4096, fmt="fp32", out="bf16"),
        # float logits of a verify batch over a slice of a vocabulary
        dict(name="product_t333_odd_e8m0", op="product", M=333, N=5003, K=6144, fmt="e8m0", out="fp32"),
        # a prompt chunk through an MLP's first projection
        dict(name="product_t8192", op="product", M=8192, N=4096, K=6144, fmt="fp32", out="bf16"),
        # a decode batch's new tokens into the cache
        dict(name="append_b16", op="append", B=16, q=1, ragged=False, len=1000, heads=32, kv=8, D=128),
        # chunks of prompts into the cache
        dict(name="append_b8_chunk", op="append", B=8, q=256, ragged=True, len=1537, heads=64, kv=8, D=128),
        # one request with a long context
        dict(name="attend_b1_long", op="attend", B=1, q=1, ragged=False, len=131000, heads=32, kv=8, D=128, mass=False),
        # a decode batch of requests of every length that feeds the eviction
        dict(name="attend_b64_mass", op="attend", B=64, q=1, ragged=False, len=8192, heads=32, kv=8, D=128, mass=True),
        # a speculative-verify batch: 32 requests of up to 4 tokens
        dict(name="attend_b32_verify", op="attend", B=32, q=4, ragged=True, len=2100, heads=16, kv=2, D=64, mass=False),
        # one request over its page budget
        dict(name="evict_b1", op="evict", B=1, len=9000, keep=100),
        # a decode batch with budgets
        dict(name="evict_b64", op="evict", B=64, len=65536, keep=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "product", "product", "append", "attend", "attend", "evict"])
    if op == "quant":
        return dict(op=op, M=_log(rng, 1, 4096), K=BLOCK * _log(rng, 1, 32), limit=rng.choice([0.0, 7.0]))
    if op == "product":
        return dict(op=op, M=_log(rng, 1, 4096), N=_log(rng, 16, 8192), K=BLOCK * _log(rng, 1, 48),
                    fmt=rng.choice(["fp32", "e8m0"]), out=rng.choice(["bf16", "fp32"]))
    if op == "evict":
        return dict(op=op, B=_log(rng, 1, 64), len=_log(rng, 64, 65536), keep=_log(rng, 4, 700))
    kv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 192, 256])
    heads = kv * rng.choice([1, 2, 4, 5, 8])
    if op == "append":
        return dict(op=op, B=_log(rng, 1, 32), q=_log(rng, 1, 256), ragged=rng.random() < 0.5,
                    len=_log(rng, 256, 4096), heads=heads, kv=kv, D=D)
    B, q = _log(rng, 1, 64), _log(rng, 1, 16)
    # bounded so that no draw reads more than the largest listed case
    most = 64 * 8192 * 8 * 128 // (B * kv * D * max(1, q // 4))
    return dict(op=op, B=B, q=q, ragged=rng.random() < 0.5, len=_log(rng, 64, max(80, min(32768, most))),
                heads=heads, kv=kv, D=D, mass=rng.random() < 0.5)


# ---- sizes that follow from a case alone -------------------------------------

def _lens(case):
    """Cached tokens and new tokens per sequence: a single request has the
    stated length, a batch is spread below it; some are empty."""
    r = random.Random(1000003 * case["B"] + case["len"])
    lens, qs = [], []
    for b in range(case["B"]):
        n = case["len"] if case["B"] == 1 or b == 0 else _log(r, max(1, case["len"] // 16), case["len"])
        q = case.get("q", 0)
        if case.get("ragged") and b > 0:
            q = r.randrange(0, q + 1)
        if b == 5:  # a padded batch row
            n = q = 0
        lens.append(max(n, q))
        qs.append(q)
    return lens, qs


def work(case):
    op = case["op"]
    if op == "quant":
        n = case["M"] * case["K"]
        return dict(bytes=n * (5 if case["limit"] else 3) + n // BLOCK, flops=n * (10 if case["limit"] else 3))
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=M * K + M * K // BLOCK + N * K + -(-N // BLOCK) * (K // BLOCK) * (4 if case["fmt"] == "fp32" else 1)
                    + M * N * (2 if case["out"] == "bf16" else 4), flops=2 * M * N * K)
    lens, qs = _lens(case)
    if op == "append":
        n = sum(qs) * case["kv"] * case["D"] * 2
        return dict(bytes=3 * n, flops=3 * n)
    if op == "attend":
        row = case["heads"] * case["D"]
        return dict(bytes=2 * case["kv"] * case["D"] * sum(n for n, q in zip(lens, qs) if q) + 4 * sum(qs) * row
                    + (8 * sum(-(-n // PAGE) for n in lens) if case["mass"] else 0),
                    flops=4 * row * sum(n * q for n, q in zip(lens, qs)))
    n = sum(-(-x // PAGE) for x in lens)
    return dict(bytes=8 * n + 12 * case["B"] * -(-case["len"] // PAGE), flops=32 * n)


# ---- inputs ------------------------------------------------------------------

def _exponent(amax):
    """The least e with amax <= 448 * 2^e, in [-127, 127]; -127 for 0."""
    m, ex = torch.frexp(amax)
    e = torch.where(m <= 0.875, ex - 9, ex - 8)
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)


def _pow2(e, dtype=torch.float32):
    """2^e, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64).to(dtype)


def _quant_last(v):
    """Codes and scale bytes of v over its last dimension (finite values)."""
    e = _exponent(v.abs().amax(-1))
    return (v * _pow2(-e, v.dtype)[..., None]).float().to(F8), (e + 127).to(torch.uint8)


def _make_pool(g, pages, kv, D):
    pool = torch.empty(pages, 2, kv, PAGE * D, dtype=torch.uint8, device=DEV)
    scale = torch.empty(pages, 2, kv, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 28) // (2 * kv * PAGE * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        v = torch.randn(n, 2, kv, PAGE * D, generator=g, device=DEV)
        v *= torch.exp(0.5 * torch.randn(n, 2, kv, 1, generator=g, device=DEV))
        c, s = _quant_last(v)
        pool[p:p + n], scale[p:p + n] = c.view(torch.uint8), s
    return pool, scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "quant":
        M, K = case["M"], case["K"]
        cols = 2 * K if case["limit"] else K
        x = torch.randn(M, cols, generator=g, device=DEV)
        x *= torch.exp(0.7 * torch.randn(1, cols, generator=g, device=DEV))  # channels of their own size
        s.update(x=(2 * x).to(torch.bfloat16), codes=torch.empty(M, K, dtype=torch.uint8, device=DEV),
                 scales=torch.empty(M, K // BLOCK, dtype=torch.uint8, device=DEV))
        return s
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        x = torch.randn(M, K, generator=g, device=DEV) * torch.exp(0.7 * torch.randn(1, K, generator=g, device=DEV))
        c, sc = _quant_last(x.to(torch.bfloat16).float().view(M, K // BLOCK, BLOCK))
        R = -(-N // BLOCK)
        w = torch.zeros(R * BLOCK, K, device=DEV)
        w[:N] = torch.randn(N, K, generator=g, device=DEV) / math.sqrt(K)
        w = w.view(R, BLOCK, K // BLOCK, BLOCK).transpose(1, 2).reshape(R, K // BLOCK, -1)
        w *= torch.exp(0.3 * torch.randn(R, K // BLOCK, 1, generator=g, device=DEV))
        if case["fmt"] == "fp32":
            ws = w.abs().amax(-1) / 448
            wc = (w / ws[..., None]).clamp(-448, 448).to(F8)
        else:
            wc, ws = _quant_last(w)
        wc = wc.view(torch.uint8).view(R, K // BLOCK, BLOCK, BLOCK).transpose(1, 2).reshape(R * BLOCK, K)[:N].contiguous()
        s.update(codes=c.view(torch.uint8).view(M, K), scales=sc, w=wc, w_scale=ws.contiguous(),
                 out=torch.empty(M, N, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device=DEV))
        if own:
            import moe_decode_layer_sigmoid_amd as md
            s["plan"] = md.ProductPlan(md.make_product_desc(N, K, M, case["fmt"], case["out"]))
        return s
    lens, qs = _lens(case)
    B, P = case["B"], -(-case["len"] // PAGE)
    i32 = dict(dtype=torch.int32, device=DEV)
    perm = torch.randperm(B * P, generator=g, device=DEV).to(torch.int32)
    s.update(table=perm.view(B, P), lens=torch.tensor(lens, **i32), P=P)
    if op == "evict":
        n = torch.tensor([-(-x // PAGE) for x in lens], device=DEV)
        mass = torch.exp(2 * torch.randn(B, P, generator=g, device=DEV))
        mass = torch.where(torch.rand(B, P, generator=g, device=DEV) < 0.1, 0.0, mass)  # pages never looked at
        s.update(mass=torch.where(torch.arange(P, device=DEV) < n[:, None], mass, 0.0), out_table=torch.empty(B, P, **i32),
                 out_lens=torch.empty(B, **i32), out_mass=torch.empty(B, P, device=DEV), freed=torch.empty(B, P, **i32),
                 n_freed=torch.empty(B, **i32))
    else:
        heads, kv, D = case["heads"], case["kv"], case["D"]
        T = sum(qs)
        starts = [0]
        for q in qs:
            starts.append(starts[-1] + q)
        pool, scale = _make_pool(g, B * P, kv, D)
        # q, k and v as they leave a fused projection, with rows behind the last sequence
        qkv = torch.randn(T + 3, (heads + 2 * kv) * D, generator=g, device=DEV)
        qkv *= torch.exp(0.5 * torch.randn(1, (heads + 2 * kv) * D, generator=g, device=DEV))
        qkv = qkv.to(torch.bfloat16)
        s.update(pool=pool, pool_scale=scale, q_start=torch.tensor(starts, **i32), T=T + 3, qmax=max(1, case["q"]),
                 q=qkv[:, :heads * D].unflatten(1, (heads, D)),
                 k=qkv[:, heads * D:(heads + kv) * D].unflatten(1, (kv, D)), v=qkv[:, (heads + kv) * D:].unflatten(1, (kv, D)),
                 out=torch.zeros(T + 3, heads, D, dtype=torch.bfloat16, device=DEV), sm_scale=1.0 / math.sqrt(D))
        if case.get("mass"):
            s.update(mass_in=torch.rand(B, P, generator=g, device=DEV) * 10, mass_out=torch.zeros(B, P, device=DEV))
    if own:
        import moe_decode_layer_sigmoid_amd as md
        heads, kv, D = case.get("heads", 1), case.get("kv", 1), case.get("D", 64)
        s["plan"] = md.CachePlan(md.make_cache_desc(heads, kv, D, pages=B * P, max_batch=B, max_pages=P, max_q=max(1, case.get("q", 1))))
    return s


# ---- the operators -----------------------------------------------------------

def _outputs(s):
    op = s["case"]["op"]
    if op == "quant":
        return dict(codes=s["codes"].view(F8), scales=s["scales"])
    if op == "append":
        return dict(pool=s["pool"].view(F8), scales=s["pool_scale"])
    if op == "evict":
        return {n: s[n] for n in ("out_table", "out_lens", "out_mass", "freed", "n_freed")}
    return {n: s[n] for n in ("out", "mass_out") if n in s}


def run(s):
    op = s["case"]["op"]
    if own:
        import moe_decode_layer_sigmoid_amd as md
        if op == "quant":
            md.quant(s["x"], s["codes"], s["scales"], limit=s["case"]["limit"] or None)
        elif op == "product":
            s["plan"].run(s["case"]["M"], codes=s["codes"], scales=s["scales"], w=s["w"], w_scale=s["w_scale"], out=s["out"])
        elif op == "append":
            s["plan"].append(s["case"]["B"], s["T"], k=s["k"], v=s["v"], pool=s["pool"], pool_scale=s["pool_scale"],
                             page_table=s["table"], seq_lens=s["lens"], q_start=s["q_start"])
        elif op == "attend":
            s["plan"].attend(s["case"]["B"], s["T"], q=s["q"], pool=s["pool"], pool_scale=s["pool_scale"], page_table=s["table"],
                             seq_lens=s["lens"], q_start=s["q_start"], out=s["out"], sm_scale=s["sm_scale"],
                             mass_in=s.get("mass_in"), mass_out=s.get("mass_out"))
        else:
            s["plan"].evict(s["case"]["B"], s["case"]["keep"], sink=SINK, recent=RECENT, page_table=s["table"], seq_lens=s["lens"],
                            mass=s["mass"], out_table=s["out_table"], out_lens=s["out_lens"], out_mass=s["out_mass"],
                            freed=s["freed"], n_freed=s["n_freed"])
    else:
        {"quant": _quant, "product": _product, "append": _append, "attend": _attend, "evict": _evict}[op](s)
    return _outputs(s)


def _quant(s):
    M, K = s["codes"].shape
    if s["case"]["limit"]:
        # in 64 bits: values next to a border between two codes or two scales
        L = s["case"]["limit"]
        g, u = s["x"][:, :K].double().clamp(max=L), s["x"][:, K:].double().clamp(-L, L)
        a = g / (1 + torch.exp(-g)) * u
    else:
        a = s["x"].float()
    c, sc = _quant_last(a.view(M, K // BLOCK, BLOCK))
    s["codes"].copy_(c.view(torch.uint8).view(M, K))
    s["scales"].copy_(sc)


def _product(s):
    M, K = s["codes"].shape
    N = s["w"].shape[0]
    x = s["codes"].view(F8).float().view(M, K // BLOCK, BLOCK) * _pow2(s["scales"].int() - 127)[..., None]
    ws = s["w_scale"] if s["case"]["fmt"] == "fp32" else _pow2(s["w_scale"].int() - 127)
    w = s["w"].view(F8).float() * ws.repeat_interleave(BLOCK, 0, output_size=ws.shape[0] * BLOCK)[:N].repeat_interleave(BLOCK, 1, output_size=K)
    s["out"].copy_(x.view(M, K) @ w.t())


def _k_tokens(k, D):
    """K codes of pages [..., 64 * D] in storage order as [..., 64, D]."""
    return k.unflatten(-1, (D // 16, PAGE, 16)).transpose(-3, -2).flatten(-2)


def _v_tokens(v, D):
    """V codes of pages [..., 64 * D] in storage order as [..., 64, D]."""
    v = v.unflatten(-1, (4, D, 4, 4))  # g, d, a, c
    return v.movedim(-3, -1).transpose(-4, -3).flatten(-4, -2)


def _k_stored(k, D):
    return k.unflatten(-1, (D // 16, 16)).transpose(-3, -2).flatten(-3)


def _v_stored(v, D):
    return v.unflatten(-2, (4, 4, 4)).transpose(-4, -3).movedim(-1, -3).flatten(-4)


def _append(s):
    case = s["case"]
    D, kv, B = case["D"], case["kv"], case["B"]
    lens, q = s["lens"].long(), (s["q_start"][1:] - s["q_start"][:-1]).long()
    past = lens - q
    I = (s["qmax"] + PAGE - 2) // PAGE + 1  # pages that qmax tokens can touch
    first = past // PAGE
    page_i = first[:, None] + torch.arange(I, device=DEV)
    # a page that gets no token stands for the sequence's first one once more
    page_i = torch.where(page_i * PAGE < lens[:, None], page_i, first[:, None]).clamp(max=s["P"] - 1)
    page = s["table"].long().gather(1, page_i)
    pos = page_i[..., None] * PAGE + torch.arange(PAGE, device=DEV)  # [B, I, 64]
    is_old = pos < past[:, None, None]
    is_new = ~is_old & (pos < lens[:, None, None])
    src = (s["q_start"][:-1].long()[:, None, None] + pos - past[:, None, None]).clamp(0, s["k"].shape[0] - 1)
    fresh = is_new[..., 0]  # the page's first token is new: its old scale says nothing
    some = is_new.any(-1)
    old = s["pool"][page]  # [B, I, 2, kv, 64 D]
    old_e = s["pool_scale"][page].int() - 127
    new = torch.stack([s["k"][src], s["v"][src]], 2).float().transpose(3, 4)  # [B, I, 2, kv, 64, D]
    old_c = torch.stack([_k_tokens(old[:, :, 0], D), _v_tokens(old[:, :, 1], D)], 2)
    m_new, m_old = is_new[:, :, None, None, :, None], is_old[:, :, None, None, :, None]
    need = _exponent(torch.where(m_new, new.abs(), 0.0).amax((-1, -2)))
    e = torch.where(fresh[:, :, None, None], need, torch.maximum(need, old_e))
    e = torch.where(some[:, :, None, None], e, old_e)
    new_c = (new * _pow2(-e)[..., None, None]).clamp(-448, 448).to(F8)
    moved = (old_c.view(F8).float() * _pow2(old_e - e)[..., None, None]).to(F8)
    c = torch.where(m_new, new_c.view(torch.uint8), torch.where(m_old, moved.view(torch.uint8), old_c))
    s["pool"][page] = torch.stack([_k_stored(c[:, :, 0], D), _v_stored(c[:, :, 1], D)], 2)
    s["pool_scale"][page] = (e + 127).to(torch.uint8)


def _attend(s):
    case = s["case"]
    B, D, kv, heads, Q, P = case["B"], case["D"], case["kv"], case["heads"], s["qmax"], s["P"]
    G = heads // kv
    lens, start = s["lens"].long(), s["q_start"].long()
    q_len = start[1:] - start[:-1]
    table = s["table"].long()
    e = _pow2(s["pool_scale"][table].int() - 127)  # [B, P, 2, kv]
    codes = s["pool"][table]
    pos = torch.arange(P * PAGE, device=DEV)
    here = (pos < lens[:, None])[:, None, :, None]
    # [B, kv, tokens, D], zero behind the sequence's last token
    k = (_k_tokens(codes[:, :, 0], D).view(F8).float() * e[:, :, 0, :, None, None]).transpose(1, 2).flatten(2, 3)
    v = (_v_tokens(codes[:, :, 1], D).view(F8).float() * e[:, :, 1, :, None, None]).transpose(1, 2).flatten(2, 3)
    del codes
    k, v = torch.where(here, k, 0.0), torch.where(here, v, 0.0)
    j = torch.arange(Q, device=DEV)
    rows = (start[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)  # [B, Q]
    q = s["q"][rows].float().unflatten(2, (kv, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, kv, G Q, D]
    sc = (q @ k.transpose(-1, -2)) * s["sm_scale"]
    seen = pos < (lens - q_len + 1)[:, None, None] + j[None, :, None]  # [B, Q, tokens]
    seen = seen & (j[None, :, None] < q_len[:, None, None]) & (pos < lens[:, None, None])
    seen = seen[:, None, None].expand(B, 1, G, Q, P * PAGE).flatten(2, 3)
    sc = torch.where(seen, sc, -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(torch.isfinite(top), top, 0.0))
    p = torch.where(seen, p, 0.0)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    o = (p @ v).unflatten(2, (G, Q)).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B, Q, heads, D]
    t = torch.arange(s["out"].shape[0], device=DEV)
    b = torch.searchsorted(start[1:].contiguous(), t, right=True).clamp(max=B - 1)
    jt = (t - start[:-1][b]).clamp(0, Q - 1)
    s["out"].copy_(torch.where((t < start[-1])[:, None, None], o[b, jt].to(torch.bfloat16), s["out"]))
    if "mass_out" in s:
        m = p.sum((1, 2)).view(B, P, PAGE).sum(-1)
        s["mass_out"].copy_(torch.where(torch.arange(P, device=DEV) * PAGE < lens[:, None], s["mass_in"] + m, s["mass_out"]))


def _evict(s):
    P, keep = s["P"], s["case"]["keep"]
    n = ((s["lens"].long() + PAGE - 1) // PAGE)[:, None]
    i = torch.arange(P, device=DEV)[None]
    key = torch.where((i < SINK) | (i >= n - RECENT), math.inf, s["mass"])
    key = torch.where(i < n, key, -1.0)
    order = torch.sort(key, dim=1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(1, order, i.expand_as(order))
    kept = (rank < torch.minimum(n, torch.full_like(n, keep))) & (i < n)
    gone = (i < n) & ~kept
    # kept pages to the front, gone pages to the front of `freed`, in order; one more column takes the rest
    to = torch.where(kept, kept.cumsum(1) - 1, P)
    to_f = torch.where(gone, gone.cumsum(1) - 1, P)
    wide = torch.full((n.shape[0], P + 1), -1, dtype=torch.int32, device=DEV)
    s["out_table"].copy_(wide.scatter(1, to, s["table"])[:, :P])
    s["freed"].copy_(wide.scatter(1, to_f, s["table"])[:, :P])
    s["out_mass"].copy_(torch.zeros(n.shape[0], P + 1, device=DEV).scatter(1, to, s["mass"])[:, :P])
    dropped = gone.sum(1)
    s["n_freed"].copy_(dropped)
    s["out_lens"].copy_(s["lens"] - PAGE * dropped)


# ---- in 64 bits --------------------------------------------------------------

def _e4m3_values():
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if c & 127 == 127 else m / 512 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _power(e):
    table = torch.tensor([2.0 ** k for k in range(-256, 257)], dtype=torch.float64, device=DEV)
    return table[e.long() + 256]


def _round_e4m3(v):
    """The e4m3 value next to v, ties to even, |v| <= 448 afterwards."""
    e = torch.frexp(v.abs().clamp(min=2.0 ** -6))[1] - 1
    step = _power(e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _scale64(amax):
    e = torch.full_like(amax, -127.0)
    for k in range(-126, 128):  # the definition, exponent by exponent
        e = torch.where(amax > 448 * 2.0 ** (k - 1), float(k), e)
    return e


def exact(case, seed):
    s = prepare(case, seed)
    op, val = case["op"], _e4m3_values()
    if op == "quant":
        M, K = s["codes"].shape
        x, L = s["x"].double(), case["limit"]
        a = torch.sigmoid(x[:, :K].clamp(max=L)) * x[:, :K].clamp(max=L) * x[:, K:].clamp(-L, L) if L else x
        a = a.view(M, -1, BLOCK)
        e = _scale64(a.abs().amax(2))
        return dict(codes=_round_e4m3(a * _power(-e)[..., None]).view(M, K), scales=(e + 127).to(torch.uint8))
    if op == "product":
        M, K = s["codes"].shape
        x = val[s["codes"].int()] * _power(s["scales"].double() - 127).repeat_interleave(BLOCK, 1)
        ws = s["w_scale"].double() if case["fmt"] == "fp32" else _power(s["w_scale"].double() - 127)
        out = torch.empty(M, case["N"], dtype=torch.float64, device=DEV)
        for n in range(0, case["N"], BLOCK):
            w = val[s["w"][n:n + BLOCK].int()] * ws[n // BLOCK].repeat_interleave(BLOCK)
            out[:, n:n + BLOCK] = x @ w.t().contiguous()
        return dict(out=out)
    lens, qs = _lens(case)
    D, kv = case.get("D"), case.get("kv")
    if op == "evict":
        outs = {n: s[n].double().cpu() if n == "out_mass" else s[n].cpu() for n in ("out_table", "out_lens", "out_mass", "freed", "n_freed")}
        for b, length in enumerate(lens):
            n = -(-length // PAGE)
            mass, ids = s["mass"][b].tolist(), s["table"][b].tolist()
            free = [i for i in range(n) if i >= SINK and i < n - RECENT]
            drop = set(sorted(free, key=lambda i: (mass[i], -i))[:max(0, n - case["keep"])])
            left, lost = [i for i in range(n) if i not in drop], sorted(drop)
            pad = s["P"] - len(left)
            outs["out_table"][b] = torch.tensor([ids[i] for i in left] + [-1] * pad, dtype=torch.int32)
            outs["out_mass"][b] = torch.tensor([mass[i] for i in left] + [0.0] * pad, dtype=torch.float64)
            outs["freed"][b] = torch.tensor([ids[i] for i in lost] + [-1] * (s["P"] - len(lost)), dtype=torch.int32)
            outs["n_freed"][b], outs["out_lens"][b] = len(lost), length - PAGE * len(lost)
        return outs
    t = torch.arange(PAGE, device=DEV)
    d = torch.arange(D, device=DEV)
    at_k = (d // 16 * PAGE * 16 + d % 16)[None] + 16 * t[:, None]  # [64, D] places in a page
    at_v = (d * 16)[None] + ((t % 16 // 4) * D * 16 + t // 16 * 4 + t % 4)[:, None]
    start = s["q_start"].tolist()
    if op == "append":
        out = val[s["pool"].int()]
        scales = s["pool_scale"].clone()
        for b, (length, q) in enumerate(zip(lens, qs)):
            past = length - q
            for pi in range(past // PAGE, -(-length // PAGE) if q else 0):
                page = int(s["table"][b, pi])
                lo, hi = max(past, pi * PAGE), min(length, (pi + 1) * PAGE)
                for kind, x, at in ((0, s["k"], at_k), (1, s["v"], at_v)):
                    new = x[start[b] + lo - past:start[b] + hi - past].double().transpose(0, 1)  # [kv, n, D]
                    e = _scale64(new.abs().amax((1, 2)))
                    was = scales[page, kind].double() - 127
                    e = e if lo == pi * PAGE else torch.maximum(e, was)
                    a = out[page, kind].clone()
                    old = at[:lo - pi * PAGE].reshape(-1)
                    a[:, old] = _round_e4m3(a[:, old] * _power(was - e)[:, None])
                    a[:, at[lo - pi * PAGE:hi - pi * PAGE].reshape(-1)] = _round_e4m3(new * _power(-e)[:, None, None]).flatten(1)
                    out[page, kind] = a
                    scales[page, kind] = (e + 127).to(torch.uint8)
        return dict(pool=out, scales=scales)
    heads = case["heads"]
    out = s["out"].double()
    outs = dict(out=out)
    if "mass_out" in s:
        outs["mass_out"] = s["mass_out"].double()
    for b, (length, q) in enumerate(zip(lens, qs)):
        n = -(-length // PAGE)
        if not n:
            continue
        ids = s["table"][b, :n].long()
        two = _power(s["pool_scale"][ids].double() - 127)
        mass = torch.zeros(n * PAGE, dtype=torch.float64, device=DEV)
        seen = torch.arange(n * PAGE, device=DEV)[None] < length - q + 1 + torch.arange(q, device=DEV)[:, None]
        for h in range(kv if q else 0):
            k = (val[s["pool"][ids, 0, h][:, at_k].int()] * two[:, 0, h, None, None]).flatten(0, 1)
            v = (val[s["pool"][ids, 1, h][:, at_v].int()] * two[:, 1, h, None, None]).flatten(0, 1)
            v[length:] = 0
            for a in range(h * (heads // kv), (h + 1) * (heads // kv)):
                sc = s["q"][start[b]:start[b + 1], a].double() @ k.t().contiguous() * s["sm_scale"]
                p = torch.softmax(sc.masked_fill(~seen, -math.inf), 1)
                out[start[b]:start[b + 1], a] = p @ v
                mass += p.sum(0)
        if "mass_out" in s:
            outs["mass_out"][b, :n] = s["mass_in"][b, :n].double() + mass.view(n, PAGE).sum(1)
    return outs
