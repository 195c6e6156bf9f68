"""The short convolution, the selective scan and the attention over shared
prefixes used together, as a stack serves and trains with them; in HIP graphs, on
streams at once, and at the ends of large arrays, on an MI355X."""
import pytest

import _selective_ref as ref
from test_gpu_cache4_shared import attention, build, i32
from test_gpu_selective_scan import made, within

torch = pytest.importorskip("torch")
import gated_delta_rule_91_amd as kda

pytestmark = pytest.mark.gpu


def gpu_random(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=gen, device="cuda")


def test_a_shared_prompt_then_own_prompts_then_steps():
    """One prompt of 45 tokens that three requests share and a request by itself: the shared prompt runs once and its
    states are copied, then the requests' own prompts as a packed batch, then steps of single tokens.  Every request is as
    over the whole of its tokens."""
    r = gpu_random(12)
    D, W, N, page, kv, heads, d, shared = 70, 4, 16, 16, 2, 8, 64, 45
    weight, bias, skip, dt_bias, A = r(D, W), r(D), r(D), r(D), -torch.exp(r(D, N))
    cache = kda.Cache4.empty(60, page, kv, d)
    free = torch.randperm(60).to(torch.int32).cuda()
    n, table = 4, i32([[-1] * 10] * 4)
    rows = {k: [[] for _ in range(n)] for k in ("u", "dt", "B", "C", "z", "conv", "out")}
    keep = lambda s, at, m, **named: [rows[k][s].append(t[..., at:at + m, :].reshape(m, -1).cpu()) for k, t in named.items()]
    prefix, offsets = i32([shared]), i32([0, 3])

    def mix(T, cu, conv_state, scan_state):
        i = dict(u=r(1, T, D), dt=r(1, T, D), B=r(1, T, N), C=r(1, T, N), z=r(1, T, D))
        i["conv"], conv_state = kda.short_conv_prefill(i["u"], weight, bias, state_in=conv_state, cu_seqlens=cu)
        i["out"], scan_state = kda.selective_scan_prefill(i["conv"], i["dt"], A, i["B"], i["C"], skip, i["z"], dt_bias, scan_state, cu)
        return i, conv_state, scan_state

    # the shared prompt, by the first request; its attention is as for any prompt
    _, _, slots, taken = kda.plan_requests(i32([0] * n), i32([shared, 0, 0, 0]), table, free, page, shared)
    free = free[int(taken):].contiguous()
    i, conv_state, scan_state = mix(shared, None, None, None)
    kda.cache4_append(cache, r(shared, kv, d), r(shared, kv, d), slots)
    for s in range(3):
        keep(s, 0, shared, **{k: v[0] for k, v in i.items()})
    zero = torch.zeros_like
    conv_state = torch.cat([conv_state] * 3 + [zero(conv_state)])
    scan_state = torch.cat([scan_state] * 3 + [zero(scan_state)])
    # the other two name its pages: whole ones are theirs too, the one in which it ends is copied
    whole = shared // page
    past = [shared] * 3 + [0]
    for s in (1, 2):
        table[s, :whole] = table[0, :whole]
        table[s, whole] = free[s - 1]
        for a in (cache.k, cache.v, cache.k_scale, cache.v_scale):
            a[int(free[s - 1])] = a[int(table[0, whole])]
    free = free[2:].contiguous()

    for new in ([20, 33, 1, 30], [1, 1, 1, 1], [1, 1, 1, 1]):
        T = sum(new)
        cu, total, slots, taken = kda.plan_requests(i32(past), i32(new), table, free, page, T)
        free = free[int(taken):].contiguous()
        if T > n:
            i, conv_state, scan_state = mix(T, cu, conv_state, scan_state)
            i = {k: v[0] for k, v in i.items()}
        else:
            i = dict(u=r(n, D), dt=r(n, D), B=r(n, N), C=r(n, N), z=r(n, D))
            i["conv"] = kda.short_conv_step(i["u"], weight, conv_state, bias)
            i["out"] = kda.selective_scan_step(i["conv"], i["dt"], A, i["B"], i["C"], scan_state, skip, i["z"], dt_bias)
        kda.cache4_append(cache, r(T, kv, d), r(T, kv, d), slots)
        q, g = r(T, heads, d), r(T, heads, d)
        out = kda.cache4_shared_attention(q, cache, table, total, prefix, offsets, cu_seqlens=cu, g=g, max_q=max(new))
        torch.cuda.synchronize()
        at, bounds, tables = 0, [0], table.tolist()
        for s, m in enumerate(new):
            keep(s, at, m, **i)
            at += m
            bounds.append(at)
        # the attention, in which the table of each request holds the prefix as well
        b = dict(c=cache, q=q, g=g, table=tables, total=total.tolist(), cu=bounds, first=[0, 0, 0, 3], before=[shared] * 3 + [0])
        want, mag, size = attention(b, d ** -0.5)
        tol = (2 * (d + 8) * size + max(b["total"]) + 24 + 1) * 2.0 ** -24 * mag + 2.0 ** -24 * want.abs() + 1e-30
        assert ((out.cpu().double() - want).abs() <= tol).all()
        past = total.tolist()
    for s in range(n):
        whole = {k: torch.cat(v[s])[None] for k, v in rows.items()}
        want = ref.conv(whole["u"], weight.cpu(), bias.cpu(), True, None)
        within(whole["conv"], want["out"], ("conv", s))
        within(conv_state[s:s + 1], want["state"], ("conv's state", s))
        want = ref.scan(whole["conv"], whole["dt"], A.cpu(), whole["B"], whole["C"], skip.cpu(), whole["z"], dt_bias.cpu())
        within(whole["out"], want["out"], ("scan", s))
        within(scan_state[s:s + 1], want["state"], ("scan's state", s))


def replays(graph, reset, outputs, expected, n=4):
    for _ in range(n):
        reset()
        torch.randn(1000, device="cuda").sum().item()      # the program's own eager work
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outputs, expected):
            assert torch.equal(a, b)


def captured(step):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    return graph, res


def test_serving_step_in_a_graph():
    """The steps and the attention captured once; lengths and prefixes change on the device."""
    r = gpu_random(3)
    n, D, W, N = 7, 130, 4, 16
    b = build([0, 4, 6], [0, 0], [450] * 4 + [240] * 2 + [150], [1] * 7, 8, 2, 128, 16, "bf16")
    total, prefix, table, offsets = i32(b["total"]), i32(b["prefix"]), i32(b["table"]), i32(b["offsets"])
    weight, A, u, dt, B, C = r(D, W), -torch.exp(r(D, N)), r(n, D).bfloat16(), r(n, D).bfloat16(), r(n, N).bfloat16(), r(n, N).bfloat16()
    conv0, scan0 = r(n, W - 1, D).bfloat16(), r(n, D, N)
    conv, scan = conv0.clone(), scan0.clone()

    def reset():
        conv.copy_(conv0)
        scan.copy_(scan0)

    def step():
        x = kda.short_conv_step(u, weight, conv)
        y = kda.selective_scan_step(x, dt, A, B, C, scan)
        return [x, y, kda.cache4_shared_attention(b["q"], b["c"], table, total, prefix, offsets, g=b["g"]), conv, scan]

    reset()
    graph, res = captured(step)
    full = b["total"]
    for before, lens in (([300, 90], full), ([200, 0], [t - 120 for t in full]), ([300, 90], full), ([0, 33], [1, 2, 3, 4, 50, 60, 70])):
        prefix.copy_(i32(before))
        total.copy_(i32(lens))
        reset()
        expected = [t.clone() for t in step()]
        torch.cuda.synchronize()
        replays(graph, reset, res, expected)


@pytest.mark.parametrize("packed", [False, True])
def test_training_pass_in_a_graph(packed):
    """The convolution and the scan forward and backward; in a packed batch with a sequence of no tokens and tokens of none."""
    r = gpu_random(5)
    B, T, D, W, N = (1 if packed else 2), 700, 130, 4, 16
    cu = i32([0, 5, 5, 400, 650]) if packed else None
    i = made(B, T, D, N, "bf16")
    weight, bias = r(D, W), r(D)
    given = dict(skip=i["skip"], z=i["z"], dt_bias=i["dt_bias"], cu_seqlens=cu)

    def step():
        x, _ = kda.short_conv_prefill(i["x"], weight, bias, cu_seqlens=cu, out=torch.zeros_like(i["x"]))
        out, state, ws = kda.selective_scan_prefill_for_backward(x, i["dt"], i["A"], i["B"], i["C"], **given, out=torch.zeros_like(x))
        g = kda.selective_scan_backward(x, i["dt"], i["A"], i["B"], i["C"], ws, **given, d_out=i["d_out"], want_dstate=False)
        h = kda.short_conv_backward(i["x"], weight, g["dx"], bias, cu_seqlens=cu, want_dstate=False)
        named = [g[k] for k in ("dA", "dskip", "ddt_bias")] + [h["dweight"], h["dbias"], state]
        tokens = [out] + [g[k] for k in ("ddt", "dB", "dC", "dz")] + [h["dx"]]
        end = T if cu is None else 650                     # tokens of no sequence are not written
        return named + [t[:, :end] for t in tokens]

    graph, res = captured(step)
    for k in range(2):
        i["x"].copy_(r(B, T, D))
        expected = [t.clone() for t in step()]
        torch.cuda.synchronize()
        replays(graph, lambda: None, res, expected)


def test_backward_twice():
    """What the forward call keeps serves a second backward, with the same results."""
    i = made(2, 900, 70, 16, "bf16")
    leaves = [i[k].requires_grad_() for k in ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias", "state")]
    weight = gpu_random(1)(70, 4).requires_grad_()
    x, _ = kda.short_conv_autograd(leaves[0], weight)
    out, state = kda.selective_scan_autograd(x, *leaves[1:])
    loss = (out.float() * i["d_out"]).sum() + (state * i["d_state"]).sum()
    first = torch.autograd.grad(loss, leaves + [weight], retain_graph=True)
    second = torch.autograd.grad(loss, leaves + [weight])
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_two_graphs_with_one_workspace():
    """Replayed in turn on a stream, each is as alone: nothing lives in a workspace from one call to the next but what the
    training pair keeps there."""
    a = build([0, 3], [200], [40, 60, 9], [1] * 3, 8, 2, 128, 16, "bf16")
    b = build([0, 2, 4], [500, 33], [7, 90, 1, 20], [1] * 4, 8, 2, 128, 16, "bf16", seed=1)
    args = [(x["q"], x["c"], i32(x["table"]), i32(x["total"]), i32(x["prefix"]), i32(x["offsets"])) for x in (a, b)]
    ws = torch.empty(max(kda.cache4_shared_attention_workspace_size(*x) for x in args), dtype=torch.uint8, device="cuda")
    s = [made(1, 3000, 70, 16, "f32"), made(2, 500, 515, 8, "bf16", seed=1)]
    given = [([x[k] for k in ("x", "dt", "A", "B", "C")], {k: x[k] for k in ("skip", "z", "dt_bias")}) for x in s]
    scan_ws = torch.empty(max(kda.selective_scan_workspace_size(kda.selective_scan_problem(*x["x"].shape, x["A"].shape[1], x["x"].dtype))
                              for x in s), dtype=torch.uint8, device="cuda")
    steps = [lambda k=k: [kda.cache4_shared_attention(*args[k], workspace=ws), *kda.selective_scan_prefill(*given[k][0], **given[k][1], workspace=scan_ws)]
             for k in range(2)]
    expected = [[t.clone() for t in step()] for step in steps]
    graphs = [captured(step) for step in steps]
    for k in (0, 1, 1, 0, 1, 0):
        torch.randn(1000, device="cuda").sum().item()
        graphs[k][0].replay()
        torch.cuda.synchronize()
        for x, y in zip(graphs[k][1], expected[k]):
            assert torch.equal(x, y)


def test_calls_on_streams_at_once():
    """Each on a stream of its own, twice one after the other: as on the current stream."""
    r = gpu_random(8)
    i = made(2, 2000, 300, 16, "bf16")
    args, given = [i[k] for k in ("x", "dt", "A", "B", "C")], {k: i[k] for k in ("skip", "z", "dt_bias")}
    weight = r(300, 4)
    b = build([0, 4], [900], [30, 60, 90, 1], [1] * 4, 8, 2, 128, 16, "f32")
    shared = (b["q"], b["c"], i32(b["table"]), i32(b["total"]), i32(b["prefix"]), i32(b["offsets"]))

    def train(stream=None):
        x, _ = kda.short_conv_prefill(i["x"], weight, stream=stream)
        out, state, ws = kda.selective_scan_prefill_for_backward(x, *args[1:], **given, stream=stream)
        g = kda.selective_scan_backward(x, *args[1:], ws, **given, d_out=i["d_out"], stream=stream)
        h = kda.short_conv_backward(i["x"], weight, g["dx"], stream=stream)
        # all of it is kept: what is freed here may go to another stream
        return [out, state, ws, x] + [t for t in (*g.values(), *h.values()) if t is not None]

    calls = [train, lambda stream=None: [kda.cache4_shared_attention(*shared, stream=stream)],
             lambda stream=None: list(kda.selective_scan_prefill(*args, **given, stream=stream)), train]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    for given_stream in (True, False):
        streams = [torch.cuda.Stream() for _ in calls]
        got = []
        for c, s in zip(calls, streams):
            if given_stream:
                got.append([c(stream=s), c(stream=s)])
            else:
                with torch.cuda.stream(s):
                    got.append([c(), c()])
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for res in g:
                for x, y in zip(res, w):
                    assert x.dtype == torch.uint8 or torch.equal(x, y)         # a workspace has gaps


def test_convolution_past_two_to_the_31_values():
    T, D, W, tail = 180000, 12288, 4, 300
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(1, T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    d_out = torch.zeros_like(x)
    d_out[:, -tail:].normal_(generator=gen)
    weight = torch.randn(D, W, generator=gen, device="cuda")
    out, state = kda.short_conv_prefill(x, weight)
    part, part_state = kda.short_conv_prefill(x[:, -tail:].contiguous(), weight, state_in=x[:, -tail - 3:-tail].contiguous())
    assert torch.equal(out[:, -tail:], part) and torch.equal(state, part_state)
    del out
    whole = kda.short_conv_backward(x, weight, d_out)
    keep = slice(T - tail - 3, T)
    pick = torch.tensor([0, 1, D // 2, D - 1], device="cuda")
    want = ref.conv(x[:, keep][..., pick].cpu(), weight[pick].cpu(), None, True, None, d_out=d_out[:, keep][..., pick].cpu())
    within(whole["dx"][:, keep][..., pick], want["dx"], "dx")


def test_scan_past_two_to_the_31_values():
    """Steps are long enough that nothing is left of a state after 150 tokens."""
    T, D, N, tail = 135000, 16384, 8, 200
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(1, T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    B, C = (torch.randn(1, T, N, generator=gen, device="cuda").bfloat16() for _ in range(2))
    A = -2.0 - torch.rand(D, N, generator=gen, device="cuda")
    out, state = kda.selective_scan_prefill(x, torch.ones_like(x), A, B, C)
    keep, pick = slice(T - tail, T), torch.tensor([0, 1, D // 2, D - 1], device="cuda")
    last = x[:, keep][..., pick]
    want = ref.scan(last.cpu(), torch.ones_like(last).cpu(), A[pick].cpu(), B[:, keep].cpu(), C[:, keep].cpu())
    within(out[:, -50:][..., pick], tuple(t[:, -50:] for t in want["out"]), "out")
    within(state[:, pick], want["state"], "state")


def test_shared_attention_in_a_cache_past_two_to_the_32_bytes():
    b = build([0, 3], [200], [40, 60, 9], [1] * 3, 8, 2, 128, 64, "bf16")
    args = lambda c, table: (b["q"], c, i32(table), i32(b["total"]), i32(b["prefix"]), i32(b["offsets"]))
    want = kda.cache4_shared_attention(*args(b["c"], b["table"]), g=b["g"])
    pages = b["c"].pages
    large = kda.Cache4.empty(2 ** 32 // (64 * 2 * 64) + 7 * pages, 64, 2, 128)
    move = lambda p: large.pages - pages + p if p < pages else p
    for name in ("k", "v", "k_scale", "v_scale"):
        getattr(large, name)[-pages:] = getattr(b["c"], name)
    # pages that do not exist lie outside the larger cache too
    table = [[move(p) if p < pages else 2 ** 31 - 1 for p in row] for row in b["table"]]
    got = kda.cache4_shared_attention(*args(large, table), g=b["g"])
    torch.cuda.synchronize()
    assert torch.equal(got, want)
