"""The operators beside the MoE layer as a decode step runs them: quantiser, q k
v projection, append, attention, eviction, output projection and the layer
itself; captured into a graph; on other streams; at offsets past 32 bits."""

import math

import numpy as np
import pytest
import torch

import layer_harness as lh
import moe_decode_layer_sigmoid_amd as md
import oracle
import ops_harness as oh
from synth import WORKLOADS, make_layer
from test_ops_gpu import check_attend, check_product, product_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Step:
    """One layer's decode step.  Sequences of `lens` cached tokens take one
    token each (`qs` tokens where given), and give back pages over `keep`."""

    HEADS, KV, D = 8, 2, 64

    def __init__(self, lens, keep, steps, qs=None):
        sh = WORKLOADS["tiny_t1"].replace(T=max(sum(qs or [1] * len(lens)), 1))
        self.inp, self.sh = make_layer(sh, seed=3), sh
        self.moe = lh.make_plan(sh)
        self.layer = lh.to_device(self.inp)
        H, heads, kv, D = sh.H, self.HEADS, self.KV, self.D
        qs = qs or [1] * len(lens)
        total = [n + steps * q for n, q in zip(lens, qs)]
        c = oh.CacheCase(7, total, qs, heads, kv, D, extra=0)
        self.B, self.T, self.P, self.keep = c.B, c.T, c.P, keep
        self.case, self.qs = c, qs
        self.dev = c.dev()
        self.dev["seq_lens"] = torch.tensor([n + q for n, q in zip(lens, qs)], dtype=torch.int32, device="cuda")
        wide = (heads + 2 * kv) * D
        i = product_inputs(1, 1, wide, H, "fp32")
        self.qkv_w, self.qkv_s = i[2].cuda(), i[3].cuda()
        i = product_inputs(2, 1, H, heads * D, "e8m0")
        self.o_w, self.o_s = i[2].cuda(), i[3].cuda()
        self.qkv_plan = md.ProductPlan(md.make_product_desc(wide, H, self.T))
        self.o_plan = md.ProductPlan(md.make_product_desc(H, heads * D, self.T, "e8m0"))
        self.plan = md.CachePlan(md.make_cache_desc(heads, kv, D, c.pages, c.B, c.P, c.max_q))
        bf = dict(dtype=torch.bfloat16, device="cuda")
        u8 = dict(dtype=torch.uint8, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        T, B, P = self.T, self.B, self.P
        self.x = torch.zeros(T, H, **bf)
        self.xc, self.xs = torch.zeros(T, H, **u8), torch.zeros(T, H // 128, **u8)
        self.qkv = torch.zeros(T, heads + 2 * kv, D, **bf)
        self.attn = torch.zeros(T, heads, D, **bf)
        self.ac, self.as_ = torch.zeros(T, heads * D, **u8), torch.zeros(T, heads * D // 128, **u8)
        self.hidden = torch.zeros(T, H, **bf)
        self.mass = torch.zeros(B, P, device="cuda")
        self.freed, self.n_freed = torch.zeros(B, P, **i32), torch.zeros(B, **i32)
        self.out, self.res = torch.zeros(T, H, **bf), torch.zeros(T, H, **bf)
        self.ids, self.w = torch.zeros(T, sh.k, **i32), torch.zeros(T, sh.k, device="cuda")

    def q_k_v(self):
        h, kv = self.HEADS, self.KV
        return self.qkv[:, :h], self.qkv[:, h:h + kv], self.qkv[:, h + kv:]

    def project(self, stream=None):
        md.quant(self.x, self.xc, self.xs, stream=stream)
        self.qkv_plan.run(self.T, codes=self.xc, scales=self.xs, w=self.qkv_w, w_scale=self.qkv_s,
                          out=self.qkv.view(self.T, -1), stream=stream)

    def append(self, stream=None):
        _, k, v = self.q_k_v()
        self.plan.append(self.B, self.T, k=k, v=v, stream=stream, **self.dev)

    def attend(self, stream=None):
        self.plan.attend(self.B, self.T, q=self.q_k_v()[0], out=self.attn, sm_scale=self.D ** -0.5,
                         mass_in=self.mass, mass_out=self.mass, stream=stream, **self.dev)

    def evict(self, stream=None):
        t, l = self.dev["page_table"], self.dev["seq_lens"]
        self.plan.evict(self.B, self.keep, sink=1, recent=1, page_table=t, seq_lens=l, mass=self.mass,
                        out_table=t, out_lens=l, out_mass=self.mass, freed=self.freed, n_freed=self.n_freed,
                        stream=stream)

    def finish(self, stream=None):
        md.quant(self.attn.view(self.T, -1), self.ac, self.as_, stream=stream)
        self.o_plan.run(self.T, codes=self.ac, scales=self.as_, w=self.o_w, w_scale=self.o_s,
                        out=self.hidden, stream=stream)
        layer = dict(self.layer, hidden=self.hidden.view(torch.int16), residual=self.x.view(torch.int16))
        self.moe.run(self.T, stream=stream, out=self.out.view(torch.int16),
                     residual_out=self.res.view(torch.int16), topk_ids=self.ids, topk_weights=self.w, **layer)

    def run(self, stream=None):
        self.project(stream)
        self.append(stream)
        self.attend(stream)
        self.evict(stream)
        self.finish(stream)

    def state(self):
        return [t.clone() for t in (self.dev["pool"], self.dev["pool_scale"], self.dev["page_table"],
                                    self.dev["seq_lens"], self.mass)]

    def restore(self, s):
        for t, x in zip((self.dev["pool"], self.dev["pool_scale"], self.dev["page_table"],
                         self.dev["seq_lens"], self.mass), s):
            t.copy_(x)

    def results(self):
        return [t.clone() for t in (self.qkv, self.attn, self.hidden, self.out, self.res, self.ids, self.freed,
                                    self.n_freed, self.dev["pool"], self.dev["pool_scale"],
                                    self.dev["page_table"], self.dev["seq_lens"], self.mass)]

    def next_token(self):
        """The next tokens' places; a sequence whose last page is full opens
        one that it gave back (here: any page that no sequence holds)."""
        table, lens = self.dev["page_table"].cpu(), self.dev["seq_lens"].cpu()
        free = [p for p in range(self.case.pages) if p not in set(table.flatten().tolist())]
        for b in range(self.B):
            lens[b] += self.qs[b]
            need = -(-int(lens[b]) // 64)
            for i in range(need):
                if table[b, i] < 0:
                    table[b, i] = free.pop()
        self.dev["page_table"].copy_(table)
        self.dev["seq_lens"].copy_(lens)

    def close(self):
        for p in (self.moe, self.qkv_plan, self.o_plan, self.plan):
            p.close()


def test_decode_steps():
    """Each operator of each step against its definition on the inputs that the
    step gives it; sequences fill pages, open new ones and give pages back."""
    steps = 4
    s = Step([62, 0, 200, 127, 320], keep=4, steps=steps)
    c, gone = s.case, 0
    g = torch.Generator().manual_seed(11)
    for step in range(steps):
        x = torch.randn(s.T, s.sh.H, generator=g).to(torch.bfloat16)
        s.x.copy_(x)
        s.project()
        codes, scales = oh.quant_ref(x)
        assert s.xs.cpu().equal(scales) and oh.same_codes(s.xc.cpu(), codes)
        check_product(codes, scales, s.qkv_w.cpu(), s.qkv_s.cpu(), s.qkv.view(s.T, -1), 2.0 ** -8)
        # the cache as it stands, for the references
        c.lens = s.dev["seq_lens"].tolist()
        c.table, c.pool, c.scale = (s.dev[n].cpu() for n in ("page_table", "pool", "pool_scale"))
        q, k, v = (t.cpu() for t in s.q_k_v())
        c.pool, c.scale = oh.append_ref(c, k, v)
        s.append()
        assert s.dev["pool_scale"].cpu().equal(c.scale) and oh.same_codes(s.dev["pool"].cpu(), c.pool)
        before = s.mass.cpu()
        s.attend()
        check = s.mass.clone()
        for b in range(s.B):
            check[b, -(-c.lens[b] // 64):] = -5
        check_attend(c, q, s.D ** -0.5, s.attn, before, check)
        ref = oh.evict_ref(c.table, c.lens, s.mass.cpu(), s.keep, 1, 1)
        s.evict()
        for name, got in (("out_table", s.dev["page_table"]), ("out_lens", s.dev["seq_lens"]),
                          ("out_mass", s.mass), ("freed", s.freed), ("n_freed", s.n_freed)):
            assert got.cpu().equal(ref[name]), (step, name)
        gone += int(s.n_freed.sum())
        s.finish()
        codes, scales = oh.quant_ref(s.attn.cpu().view(s.T, -1))
        assert s.as_.cpu().equal(scales) and oh.same_codes(s.ac.cpu(), codes)
        check_product(codes, scales, s.o_w.cpu(), s.o_s.cpu(), s.hidden, 2.0 ** -8)
        s.inp.hidden = s.hidden.view(torch.int16).cpu().numpy().view(np.uint16)
        s.inp.residual = s.x.view(torch.int16).cpu().numpy().view(np.uint16)
        ref = oracle.moe_layer(s.inp, forced_ids=s.ids.cpu().numpy())
        lh.assert_close(lh.bf16_to_np(s.out.view(torch.int16)), ref["out"], "out")
        s.next_token()
    assert gone >= 2
    s.close()


@pytest.mark.parametrize("qs", [None, [3, 0, 1, 4]])
def test_captured_step_replays(qs):
    """The whole step as one graph, replayed on other tokens and caches with
    eager steps between, gives the eager step's bits each time."""
    s = Step([100, 70, 300, 500], keep=5, steps=1, qs=qs)
    g = torch.Generator().manual_seed(5)
    start = s.state()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.run()
    torch.cuda.synchronize()
    for _ in range(4):
        x = torch.randn(s.T, s.sh.H, generator=g).to(torch.bfloat16).cuda()
        s.x.copy_(x)
        s.restore(start)
        s.run()
        torch.cuda.synchronize()
        eager = s.results()
        s.restore(start)
        for t in (s.qkv, s.attn, s.hidden, s.out):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, s.results()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    s.close()


def test_two_plans_at_once_on_two_streams():
    """Plans have their own workspaces: split products and long attentions of
    two plans, each on a stream of its own at the same time, give the bits that
    they give alone."""
    case = oh.CacheCase(4, [5000, 900], [1, 2], 8, 2, 64)
    q = case.rows(8)
    parts = product_inputs(3, 20, 300, 6144, "fp32")
    both = []
    for i in range(2):
        dev = case.dev()
        cplan = md.CachePlan(md.make_cache_desc(8, 2, 64, case.pages, case.B, case.P, case.max_q))
        pplan = md.ProductPlan(md.make_product_desc(300, 6144, 20))
        p = [t.cuda() for t in parts]
        out = torch.zeros(case.T, 8, 64, dtype=torch.bfloat16, device="cuda")
        mass = torch.zeros(case.B, case.P, device="cuda")
        y = torch.zeros(20, 300, dtype=torch.bfloat16, device="cuda")
        qd = (q * (i + 1)).cuda()

        def run(stream, cplan=cplan, pplan=pplan, p=p, out=out, mass=mass, y=y, qd=qd, dev=dev):
            for _ in range(5):
                cplan.attend(case.B, case.T, q=qd, out=out, sm_scale=0.1, mass_out=mass, stream=stream, **dev)
                pplan.run(20, codes=p[0], scales=p[1], w=p[2], w_scale=p[3], out=y, stream=stream)

        run(None)
        torch.cuda.synchronize()
        both.append((run, (out, mass, y), [t.clone() for t in (out, mass, y)], (cplan, pplan)))
        for t in (out, mass, y):
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for (run, *_), st in zip(both, streams):
        run(st if st is streams[0] else st.cuda_stream)  # a Stream, or its handle
    torch.cuda.synchronize()
    for _, got, alone, plans in both:
        for a, b in zip(got, alone):
            assert a.equal(b)
        for p in plans:
            p.close()


def test_pages_past_four_gigabytes():
    """Pages whose codes lie past 2^32 bytes of the pool."""
    case = oh.CacheCase(9, [200, 65, 1], [1, 3, 1], 4, 2, 256, spare=0)
    per_page = 2 * 2 * 64 * 256
    first = (1 << 32) // per_page + 1
    pool = torch.empty(first + case.pages, 2, 2, 64 * 256, dtype=torch.uint8, device="cuda")
    scale = torch.empty(first + case.pages, 2, 2, dtype=torch.uint8, device="cuda")
    pool[first:], scale[first:] = case.pool.cuda(), case.scale.cuda()
    dev = dict(case.dev(), pool=pool, pool_scale=scale)
    dev["page_table"] = torch.where(dev["page_table"] >= 0, dev["page_table"] + first, dev["page_table"])
    plan = md.CachePlan(md.make_cache_desc(4, 2, 256, first + case.pages, case.B, case.P, case.max_q))
    q, k, v = case.rows(4), case.rows(2, 3.0), case.rows(2)
    plan.append(case.B, case.T, k=k.cuda(), v=v.cuda(), **dev)
    case.pool, case.scale = oh.append_ref(case, k, v)
    assert scale[first:].cpu().equal(case.scale) and oh.same_codes(pool[first:].cpu(), case.pool)
    out = torch.full((case.T, 4, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    plan.attend(case.B, case.T, q=q.cuda(), out=out, sm_scale=1 / 16, **dev)
    check_attend(case, q, 1 / 16, out)
    plan.close()


def test_pages_held_twice():
    """Sequences that share pages, and one that holds a page twice."""
    case = oh.CacheCase(13, [200, 200, 256], [1, 1, 2], 6, 2, 128)
    case.table[1, :3] = case.table[0, :3]
    case.table[2, 2] = case.table[2, 0]
    q, dev = case.rows(6), case.dev()
    plan = md.CachePlan(md.make_cache_desc(6, 2, 128, case.pages, case.B, case.P, case.max_q))
    out = torch.zeros(case.T, 6, 128, dtype=torch.bfloat16, device="cuda")
    mass_in = torch.rand(case.B, case.P, generator=case.g)
    mass = torch.full((case.B, case.P), -5.0, device="cuda")
    plan.attend(case.B, case.T, q=q.cuda(), out=out, sm_scale=0.09, mass_in=mass_in.cuda(), mass_out=mass, **dev)
    check_attend(case, q, 0.09, out, mass_in, mass)
    plan.close()


def test_products_and_rows_past_four_gigabytes():
    """Outputs past 2^32 bytes, and quantised rows that far apart."""
    M, N, K = 60000, 40000, 128
    codes, scales, w, ws = product_inputs(6, 64, N, K, "fp32")
    rep = torch.arange(M) % 64
    plan = md.ProductPlan(md.make_product_desc(N, K, M))
    out = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    plan.run(M, codes=codes[rep].cuda(), scales=scales[rep].cuda(), w=w.cuda(), w_scale=ws.cuda(), out=out)
    check_product(codes, scales, w, ws, out[:64], 2.0 ** -8)
    # every row has its first 64 rows' twin
    for m0 in range(64, M, 64 * 100):
        m1 = min(M, m0 + 6400)
        want = out[:64].repeat((m1 - m0 + 63) // 64, 1)[:m1 - m0]
        assert out[m0:m1].equal(want), m0
    plan.close()
    del out, want
    x = torch.empty(2100, 1 << 20, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn(2100, 256, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[:, 64:320] = rows.cuda()
    c = torch.zeros(2100, 256, dtype=torch.uint8, device="cuda")
    s = torch.zeros(2100, 2, dtype=torch.uint8, device="cuda")
    md.quant(x[:, 64:320], c, s)
    rc, rs = oh.quant_ref(rows)
    assert s.cpu().equal(rs) and oh.same_codes(c.cpu(), rc)


def test_tensors_that_are_refused():
    """What the binding checks of tensors: types, shapes, strides, devices."""
    case = oh.CacheCase(2, [70, 20], [1, 1], 4, 2, 64)
    dev = case.dev()
    plan = md.CachePlan(md.make_cache_desc(4, 2, 64, case.pages, case.B, case.P, 1))
    q, out = case.rows(4).cuda(), torch.zeros(case.T, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = case.rows(2).cuda()
    B, T = case.B, case.T

    def refused(f, **kw):
        with pytest.raises(md.MoeDecodeError) as e:
            f(**kw)
        assert e.value.code == md.ERR_INVALID_ARG

    def attend(**kw):
        plan.attend(**{**dict(B=B, T=T, q=q, out=out, sm_scale=1.0, **dev), **kw})

    def append(**kw):
        plan.append(**{**dict(B=B, T=T, k=k, v=k, **dev), **kw})

    bufs = dict(page_table=dev["page_table"], seq_lens=dev["seq_lens"], mass=torch.zeros(B, case.P, device="cuda"),
                out_table=dev["page_table"], out_lens=dev["seq_lens"], out_mass=torch.zeros(B, case.P, device="cuda"),
                freed=torch.zeros_like(dev["page_table"]), n_freed=torch.zeros_like(dev["seq_lens"]))

    def evict(**kw):
        plan.evict(**{**dict(B=B, keep=3, sink=1, recent=1, **bufs), **kw})

    attend()
    append()
    evict(keep=2)
    for f in (attend, append):
        refused(f, B=B + 1)
        refused(f, B=-1)
        refused(f, T=T + 1)
        refused(f, pool=dev["pool"].cpu())
        refused(f, pool=dev["pool"][:-1])
        refused(f, pool_scale=dev["pool_scale"].int())
        refused(f, page_table=dev["page_table"].long())
        refused(f, page_table=dev["page_table"][:1])
        refused(f, page_table=dev["page_table"].t().contiguous().t())
        refused(f, seq_lens=dev["seq_lens"][:1])
        refused(f, q_start=dev["q_start"][:B])
    refused(attend, q=q.float())
    refused(attend, q=q[:, :2])
    refused(attend, q=q.transpose(1, 2).contiguous().transpose(1, 2))
    refused(attend, q=q.cpu())
    refused(attend, out=q)  # the output over the queries
    refused(attend, out=out[:, :, :32])
    refused(attend, sm_scale=math.inf)
    refused(attend, sm_scale=1e39)
    refused(attend, mass_in=bufs["mass"])
    refused(attend, mass_out=bufs["mass"].double())
    refused(append, k=k[:, :1])
    refused(append, v=k.half())
    refused(evict, keep=1)
    refused(evict, keep=1 << 40)
    refused(evict, recent=0)
    refused(evict, freed=bufs["freed"][:, :1])
    refused(evict, n_freed=bufs["n_freed"].long())
    plan.close()
    refused(attend)  # a closed plan

    codes, scales, w, ws = (t.cuda() for t in product_inputs(8, 5, 48, 256, "fp32"))
    y = torch.zeros(5, 48, dtype=torch.bfloat16, device="cuda")
    pplan = md.ProductPlan(md.make_product_desc(48, 256, 5))

    def product(**kw):
        pplan.run(**{**dict(M=5, codes=codes, scales=scales, w=w, w_scale=ws, out=y), **kw})

    product()
    product(codes=codes.view(torch.float8_e4m3fn))
    refused(product, M=6)
    refused(product, codes=codes[:4])
    refused(product, codes=codes.to(torch.int16))
    refused(product, scales=scales.float())
    refused(product, w=w[:40])
    refused(product, w_scale=ws.to(torch.uint8))
    refused(product, out=y.float())
    refused(product, out=y.t().contiguous().t())
    refused(product, out=y[:, :47])
    pplan.close()
    refused(product)

    x = torch.zeros(5, 256, dtype=torch.bfloat16, device="cuda")
    refused(md.quant, x=x.float(), codes=codes, scales=scales)
    refused(md.quant, x=x[:4], codes=codes, scales=scales)
    refused(md.quant, x=x, codes=codes, scales=scales, limit=1.0)  # no up half
    refused(md.quant, x=x, codes=codes, scales=scales, limit=0.0)
    refused(md.quant, x=x, codes=codes.cpu(), scales=scales)
    refused(md.quant, x=x, codes=codes, scales=scales[:, :1])
    refused(md.quant, x=x.t().contiguous().t(), codes=codes, scales=scales)
