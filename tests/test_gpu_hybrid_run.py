"""The operators beside KDA used together, as a hybrid stack serves and trains
with them, and in HIP graphs, on an MI355X."""
import math

import pytest

import _hybrid_ref as ref

torch = pytest.importorskip("torch")
import gated_delta_rule_91_amd as kda

pytestmark = pytest.mark.gpu
FLOOR = -0.5


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_prompts_then_steps():
    """Two prompts of different lengths, then decode steps of both and a third request, by one plan a step: the offsets
    feed KDA and the recurrence, the tables and slots the cache and the attention."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    n, page, kv, heads, d, D = 3, 16, 2, 4, 64, 96
    cache = kda.Cache4.empty(40, page, kv, d)
    table, free = i32([[-1] * 8] * n), torch.randperm(40, generator=gen, device="cuda").to(torch.int32)
    lens = [0] * n
    rec_state, kda_state = torch.zeros(n, D, device="cuda"), torch.zeros(n, 2, d, d, device="cuda")
    xs, las, ks, vs = ([[] for _ in range(n)] for _ in range(4))
    for new in ([37, 70, 0], [1, 1, 20], [1, 0, 1], [1, 1, 1]):
        T = sum(new)
        cu, total, slots, taken = kda.plan_requests(i32(lens), i32(new), table, free, page, T)
        free = free[int(taken):].contiguous()
        # KDA and the recurrence over the packed batch, their states carried
        q, k, v, g = (r(1, T, 2, d).bfloat16() for _ in range(4))
        _, kda_state = kda.varlen_prefill(q, k, v, -torch.rand(1, T, 2, d, generator=gen, device="cuda"),
                                          torch.rand(1, T, 2, generator=gen, device="cuda"), g, -0.1, cu, state_in=kda_state)
        x, la = r(1, T, D), -torch.rand(1, T, D, generator=gen, device="cuda")
        out, rec_state = kda.recurrence_prefill(x, la, FLOOR, state_in=rec_state, cu_seqlens=cu)
        # the attention layer: new rows into the cache, then over it
        ak, av, aq = r(T, kv, d), r(T, kv, d), r(T, heads, d)
        kda.cache4_append(cache, ak, av, slots)
        att = kda.cache4_attention(aq, cache, table, total, cu_seqlens=cu, max_q=max(new))
        torch.cuda.synchronize()
        at = 0
        for s, m in enumerate(new):
            for store, t in ((xs, x[0]), (las, la[0]), (ks, ak), (vs, av)):
                store[s].append(t[at:at + m].cpu())
            # the recurrence goes on as over the whole of its tokens
            h = ref.recurrence(torch.cat(xs[s])[None], torch.cat(las[s])[None], FLOOR, None, None)
            if m:
                assert torch.allclose(out[0, at:at + m].cpu().double(), h["out"][0, -m:], rtol=0, atol=(3 * 150 + 16) * 2.0 ** -24 * float(h["h"].abs().max()))
            k4, v4 = (ref.values(ref.packed(c), sc) for c, sc in (ref.quantized(torch.cat(t)) for t in (ks[s], vs[s])))
            for i in range(m):
                end = lens[s] + i + 1
                for head in range(heads):
                    kk, vv = k4[:end, head // 2], v4[:end, head // 2]
                    qq = aq[at + i, head].cpu().double()
                    p = torch.softmax(kk @ qq / math.sqrt(d), 0)
                    size = float((kk.abs() @ qq.abs()).max()) / math.sqrt(d)
                    tol = (2 * (d + 8) * size + end + 16 + 2) * 2.0 ** -24 * (p @ vv.abs())
                    assert ((att[at + i, head].cpu().double() - p @ vv).abs() <= tol).all()
            at += m
        lens = total.tolist()
    assert torch.isfinite(kda_state).all()


def _replays(graph, reset, outputs, expected, n=4):
    for _ in range(n):
        reset()
        torch.randn(1000, device="cuda").sum().item()      # the program's own eager work
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outputs(), expected):
            assert torch.equal(a, b)


def test_serving_step_in_a_graph():
    """Plan, append, attention and the recurrence's step captured once; lengths change on the device."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    n, page, kv, heads, d, D = 5, 16, 2, 8, 128, 70
    cache = kda.Cache4.empty(200, page, kv, d)
    pool = torch.randperm(200, generator=gen, device="cuda").to(torch.int32)
    table0 = i32([[-1] * 60] * n)
    for s in range(n):
        table0[s, :30] = pool[30 * s:30 * s + 30]
    free = pool[150:].contiguous()
    k0, v0 = (torch.randint(0, 256, cache.k.shape, generator=gen, device="cuda").to(torch.uint8) for _ in range(2))
    cache.k_scale.fill_(125)
    cache.v_scale.fill_(124)
    past, new, table = i32([0] * n), i32([1] * n), table0.clone()
    k, v, q, g = r(n, kv, d).bfloat16(), r(n, kv, d).bfloat16(), r(n, heads, d).bfloat16(), r(n, heads, d).bfloat16()
    x, la, s0 = r(n, D).bfloat16(), -torch.rand(n, D, generator=gen, device="cuda"), r(n, D)
    state = s0.clone()

    def reset():
        cache.k.copy_(k0)
        cache.v.copy_(v0)
        table.copy_(table0)
        state.copy_(s0)

    def step():
        cu, total, slots, taken = kda.plan_requests(past, new, table, free, page, n)
        kda.cache4_append(cache, k, v, slots)
        att = kda.cache4_attention(q, cache, table, total, g=g)
        out = kda.recurrence_step(x, la, state, FLOOR)
        return cu, total, slots, taken, att, out, state, table, cache.k, cache.v

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        reset()
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    reset()
    with torch.cuda.graph(graph):
        res = step()
    for lens in ([0, 5, 16, 480, 31], [300, 479, 1, 15, 64]):
        past.copy_(i32(lens))
        reset()
        expected = [t.clone() for t in step()]
        torch.cuda.synchronize()
        _replays(graph, reset, lambda: res, expected)


def test_training_pass_in_a_graph():
    gen = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    B, T, D = 2, 1500, 130
    x, g, d_out = (r(B, T, D).bfloat16() for _ in range(3))
    la, s0, ds = -torch.rand(B, T, D, generator=gen, device="cuda"), r(B, D), r(B, D)

    def step():
        out, state, ws = kda.recurrence_prefill_for_backward(x, la, FLOOR, g=g, state_in=s0)
        b = kda.recurrence_backward(x, la, FLOOR, ws, g=g, state_in=s0, d_out=d_out, d_state=ds)
        return [out, state, b["dx"], b["dlog_alpha"], b["dg"], b["dstate0"]]

    expected = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    _replays(graph, lambda: None, lambda: res, expected)


def test_other_streams_and_calls_at_once():
    """The same calls on two streams at once give what they give alone."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    jobs = []
    for T in (3000, 2900):
        x, la, g = r(1, T, 256).bfloat16(), -torch.rand(1, T, 256, generator=gen, device="cuda"), r(1, T, 256).bfloat16()
        c = kda.Cache4.empty(200, 16, 2, 64)
        k = r(T, 2, 64)
        kda.cache4_append(c, k, -k, torch.arange(T, device="cuda"))
        q, table = r(1, 8, 64), torch.arange(200, dtype=torch.int32, device="cuda")[None]
        jobs.append((x, la, g, c, q, table, i32([T])))

    def go(j, stream=None):
        x, la, g, c, q, table, total = j
        out, state = kda.recurrence_prefill(x, la, FLOOR, g=g, stream=stream)
        return out, state, kda.cache4_attention(q, c, table, total, stream=stream)

    alone = []
    for j in jobs:
        alone.append(go(j))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        outs = [None, None]
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            outs[i] = go(jobs[i], stream=s)
        torch.cuda.synchronize()
        for got, want in zip(outs, alone):
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_requests_that_were_cut_off():
    """More new tokens than rows: the offsets tell on the device, and the rows that are left attend as they would in a
    step that brings them alone."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    page, kv, heads, d = 16, 2, 4, 64
    past, new, kept = [10, 30, 3], [5, 20, 4], [5, 3, 0]
    pk, pv = ([r(p, kv, d) for p in past] for _ in range(2))
    k, v, q = r(8, kv, d), r(8, kv, d), r(8, heads, d)
    outs = []
    for lens in (new, kept):
        cache = kda.Cache4.empty(20, page, kv, d)
        for t in (cache.k_scale, cache.v_scale):
            t.fill_(255)                                  # what no token has written stands for NaN
        table, free, none = i32([[-1] * 5] * 3), torch.arange(20, dtype=torch.int32, device="cuda"), i32([0] * 3)
        _, _, slots, taken = kda.plan_requests(none, i32(past), table, free, page, sum(past))
        kda.cache4_append(cache, torch.cat(pk), torch.cat(pv), slots)
        cu, total, slots, more = kda.plan_requests(i32(past), i32(lens), table, free[int(taken):].contiguous(), page, 8)
        kda.cache4_append(cache, k, v, slots)
        assert (cu.diff() < i32(lens)).tolist() == [a < b for a, b in zip(kept, lens)]
        total = i32(past) + cu.diff()
        assert total.tolist() == [p + m for p, m in zip(past, kept)]
        outs.append(kda.cache4_attention(q, cache, table, total, cu_seqlens=cu, max_q=5))
    torch.cuda.synchronize()
    assert torch.isfinite(outs[0]).all() and torch.equal(*outs)
