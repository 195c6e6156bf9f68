"""More operators of a hybrid stack beside KDA, as measured workloads.

A recurrent mixer sees its inputs through a short causal convolution, a hybrid
stack holds selective state spaces beside its attention layers, and the
requests that such a stack serves share long prefixes: their recurrent states
are copied, their cached keys and values read once for all.  The operators are

    conv        a causal convolution over a few tokens of each channel, with
                bias and SiLU, over uniform and packed batches
    conv-train  the same with its gradients
    conv-step   the same for one token of each sequence, the window in place
    scan        a selective state space of N states a channel,
                    h_t = exp(delta_t A) h_(t-1) + delta_t x_t B_t
                    out_t = (C_t . h_t + skip x_t) silu(z_t)
                with delta = softplus(dt + dt_bias)
    scan-train  the same with its gradients
    scan-step   the same for one token of each sequence, the state in place
    shared      causal grouped-query attention over the 4-bit paged cache for
                groups of requests that share their first tokens

`own` false: `run` computes the plain forms below, elementary torch operations
in 32 bits, the state space in 64.  `own` true: `run` makes the framework's
calls.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 32            # channels of the cache that share a scale


# ---- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # queries, keys and values of the 64K prefill at once: 3 x 32 heads of 128
        dict(name="conv-64k", op="conv", rows=1, tokens=65536, requests=0, width=12288, taps=4, io="bf16", bias=False, silu=True),
        # a packed batch in 32 bits of an odd width
        dict(name="conv-packed-f32", op="conv", rows=1, tokens=16384, requests=24, width=515, taps=3, io="f32", bias=True, silu=False),
        # a training step: 4 x 4096 tokens, 3 x 16 heads of 128
        dict(name="conv-train", op="conv-train", rows=4, tokens=4096, requests=0, width=6144, taps=4, io="bf16", bias=True, silu=True),
        # one token of each of 8 sequences: latency
        dict(name="conv-step", op="conv-step", rows=8, width=12288, taps=4, io="bf16", bias=True, silu=True),
        # the 64K prefill, as wide as 16 heads of 128
        dict(name="scan-64k", op="scan", rows=1, tokens=65536, requests=0, width=2048, states=16, io="bf16", gate=True, skip=True),
        # a packed batch in 32 bits of an odd width
        dict(name="scan-packed-f32", op="scan", rows=1, tokens=16384, requests=24, width=515, states=8, io="f32", gate=False, skip=True),
        # a training step: 4 x 4096 tokens, as wide as 16 heads of 128
        dict(name="scan-train", op="scan-train", rows=4, tokens=4096, requests=0, width=2048, states=16, io="bf16", gate=True, skip=True),
        # one token of each of 256 sequences, as wide as 32 heads of 128
        dict(name="scan-step", op="scan-step", rows=256, width=4096, states=16, io="bf16", gate=True, skip=True),
        # four requests on a short instruction: latency
        dict(name="shared-few", op="shared", groups=1, requests=4, prefix=1024, most_own=100, new=1, heads=32, kv_heads=8, d=128, page=64, io="bf16", gate=True),
        # a decode step of a full serving batch whose requests share their instructions
        dict(name="shared-step", op="shared", groups=1, requests=256, prefix=8192, most_own=1000, new=1, heads=32, kv_heads=8, d=128, page=64, io="bf16", gate=True),
        # a few groups, six heads to a shared one, 32-bit activations
        dict(name="shared-groups-f32", op="shared", groups=5, requests=48, prefix=20000, most_own=700, new=1, heads=24, kv_heads=4, d=64, page=16, io="f32", gate=False),
        # prompts on a long document that is cached already
        dict(name="shared-prompts", op="shared", groups=1, requests=4, prefix=65536, most_own=1000, new=500, heads=32, kv_heads=8, d=128, page=64, io="bf16", gate=True),
    ]


def _log_uniform(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["conv", "conv-train", "conv-step", "scan", "scan", "scan-train", "scan-step", "shared", "shared", "shared"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "shared":
        c = dict(op=op, groups=_log_uniform(rng, 1, 12), kv_heads=rng.choice([1, 2, 3, 4, 8]), d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128, 256]), io=io, gate=rng.random() < 0.6)
        c["heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 6, 8])
        c["requests"] = _log_uniform(rng, c["groups"], 300)
        c["new"] = 1 if rng.random() < 0.6 else _log_uniform(rng, 2, max(2, 2000 // c["requests"]))
        c["most_own"] = c["new"] + _log_uniform(rng, 1, 1500)
        # scores of the plain form, which holds them
        most = 3000000000 // (c["heads"] * c["requests"] * c["new"] * max(1, c["groups"] // 2))
        c["prefix"] = _log_uniform(rng, 16, max(16, min(100000, most)))
        return c
    width = _log_uniform(rng, 16, 6000)
    if rng.random() < 0.5:       # whole vectors, as models have them
        width = max(64, width // 64 * 64)
    c = dict(op=op, width=width, io=io)
    if op.startswith("conv"):
        c.update(taps=rng.choice([2, 3, 4, 4]), bias=rng.random() < 0.5, silu=rng.random() < 0.7)
        cells = width
    else:
        c.update(states=rng.choice([8, 16, 16, 32]), gate=rng.random() < 0.7, skip=rng.random() < 0.7)
        cells = width * c["states"]
    if op.endswith("step"):
        return dict(c, rows=_log_uniform(rng, 1, 400))
    most = {"conv": 400, "conv-train": 90, "scan": 1500, "scan-train": 400}[op] * 1000000 // cells
    tokens = _log_uniform(rng, 1, min(60000, most))
    if rng.random() < 0.5:
        return dict(c, rows=1, tokens=tokens, requests=_log_uniform(rng, 1, min(200, tokens)))
    return dict(c, rows=_log_uniform(rng, 1, max(1, min(64, most // tokens))), tokens=tokens, requests=0)


def _lengths(n, longest, shortest, salt):
    """n ragged lengths that go by the sizes alone, the first the longest."""
    rng = random.Random(salt * 1000003 + n * 8191 + longest)
    return [longest] + [_log_uniform(rng, shortest, longest) if longest > shortest else shortest for _ in range(n - 1)]


def _cumulative(lengths):
    cu = [0]
    for m in lengths:
        cu.append(cu[-1] + m)
    return cu


def _cuts(n, total, salt, least=0):
    """Cumulative offsets of n ragged parts of `total`, each at least `least`."""
    rng = random.Random(salt * 1000003 + n * 8191 + total)
    free = total - n * least
    cuts = [0] + sorted(rng.randrange(free + 1) for _ in range(n - 1)) + [free]
    return [c + i * least for i, c in enumerate(cuts)]


def _offsets(c):
    """Cumulative offsets of the sequences over the rows laid end to end."""
    if c.get("requests"):
        return _cuts(c["requests"], c["tokens"], 5)
    return [r * c["tokens"] for r in range(c["rows"] + 1)]


def _shared_lengths(c):
    """(first request of each group, prefix of each group, own tokens of each request, new ones among these)."""
    own_lens = _lengths(c["requests"], c["most_own"], 1, 3)
    new = [min(o, m) for o, m in zip(own_lens, _lengths(c["requests"], c["new"], 1, 4))]
    return _cuts(c["groups"], c["requests"], 6, 1), _lengths(c["groups"], c["prefix"], max(1, c["prefix"] // 4), 7), own_lens, new


def _pages(tokens, page):
    return (tokens + page - 1) // page


# ---- inputs -----------------------------------------------------------------------------------

def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype).cuda()


def _cache_pair(gen, pages, page, heads, d):
    """Codes and scales of normal values, as a cache holds them."""
    codes = torch.empty(pages, heads, page, d // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, heads, page, d // GROUP, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (heads * page * d))
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for p in range(0, pages, step):
        x = torch.randn(min(step, pages - p), heads, page, d // GROUP, GROUP, generator=gen, device="cuda")
        e = torch.frexp(x.abs().amax(-1))[1] - 3
        code = torch.bucketize(torch.ldexp(x.abs(), -e[..., None]), edges) + 8 * (x < 0)
        code = code.to(torch.uint8).flatten(-2)
        codes[p:p + step], scales[p:p + step] = code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)
    return codes, scales


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    op, io = c["op"], DTYPES[c["io"]]
    s = dict(op=op)
    if op == "shared":
        first, prefix, own_lens, new = _shared_lengths(c)
        page, heads, d = c["page"], c["kv_heads"], c["d"]
        group = [j for j in range(c["groups"]) for _ in range(first[j], first[j + 1])]
        total = [prefix[j] + o for j, o in zip(group, own_lens)]
        whole = [prefix[j] // page for j in group]                    # pages that a request has from its group
        fresh = [_pages(t, page) - w for t, w in zip(total, whole)]
        pages = sum(p // page for p in prefix) + sum(fresh)
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).tolist()
        shared = [[order.pop() for _ in range(p // page)] for p in prefix]
        rows = [shared[j] + [order.pop() for _ in range(f)] for j, f in zip(group, fresh)]
        width = max(len(r) for r in rows)
        cache = {}
        cache["k"], cache["k_scale"] = _cache_pair(gen, pages, page, heads, d)
        cache["v"], cache["v_scale"] = _cache_pair(gen, pages, page, heads, d)
        T = sum(new)
        return dict(s, q=(1.5 * normal(T, c["heads"], d)).to(io), g=normal(T, c["heads"], d, dtype=io) if c["gate"] else None, cache=cache,
                    table=_ints([r + [-1] * (width - len(r)) for r in rows]), total=_ints(total), prefix=_ints(prefix), first=_ints(first),
                    cu=_ints(_cumulative(new)) if c["new"] > 1 else None, most_new=max(new), most_prefix=max(prefix), most_own=max(own_lens),
                    most_rows=max(sum(new[a:b]) for a, b in zip(first, first[1:])))
    B, T, D = c["rows"], c.get("tokens", 1), c["width"]
    step = op.endswith("step")
    shape = (B, D) if step else (B, T, D)
    n = c.get("requests") or B
    s["x"] = normal(*shape, dtype=io)
    if not step:
        s["cu"] = _ints(_offsets(c)) if c["requests"] else None
    if op.startswith("conv"):
        W = c["taps"]
        s["weight"] = normal(D, W) / math.sqrt(W)
        s["bias"] = 0.2 * normal(D) if c["bias"] else None
        s["silu"] = c["silu"]
        s["state"] = normal(n, W - 1, D, dtype=io)
        if op == "conv-train":
            s["d_out"], s["d_state"] = normal(*shape, dtype=io), normal(n, W - 1, D, dtype=io)
        return s
    N = c["states"]
    # steps from a thousandth to a tenth, states that fade at speeds from 1 to N
    start = torch.exp(uniform(D) * math.log(100) + math.log(0.001))
    s["dt_bias"] = start + torch.log(-torch.expm1(-start))
    s["dt"] = (0.5 * normal(*shape)).to(io)
    s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(0.2 * normal(D, N))
    s["B"], s["C"] = normal(*shape[:-1], N, dtype=io), normal(*shape[:-1], N, dtype=io)
    s["skip"] = normal(D) if c["skip"] else None
    s["z"] = normal(*shape, dtype=io) if c["gate"] else None
    s["state"] = 0.3 * normal(n, D, N)
    if op == "scan-train":
        s["d_out"], s["d_state"] = normal(*shape, dtype=io), normal(n, D, N)
    return s


# ---- plain forms ------------------------------------------------------------------------------

def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _spans(s):
    """Offsets of the sequences over the rows laid end to end."""
    if s["cu"] is not None:
        return s["cu"].long()
    B, T = s["x"].shape[:2]
    return torch.arange(B + 1, device="cuda") * T


def _window(s):
    """(rows with each sequence's window put before it, places of the tokens among them, places of the windows, of the last inputs)."""
    cu, before = _spans(s), s["state"].shape[1]
    x = s["x"].reshape(-1, s["x"].shape[-1])
    t = torch.arange(len(x), device="cuda")
    seq = torch.searchsorted(cu[1:], t, right=True)
    at = t + (seq + 1) * before
    i = torch.arange(before, device="cuda")
    head = (cu[:-1] + torch.arange(len(cu) - 1, device="cuda") * before)[:, None] + i
    tail = (cu[1:] + torch.arange(len(cu) - 1, device="cuda") * before)[:, None] + i
    rows = torch.zeros(len(x) + head.numel(), x.shape[1], device="cuda")
    rows[at] = x.float()
    rows[head] = s["state"].float()
    return rows, at, head, tail


def _before_silu(s, rows):
    """The convolution at every row that has a whole window, rows of windows among them."""
    w, W = s["weight"], s["weight"].shape[1]
    y = sum(w[:, j] * rows[j:len(rows) - W + 1 + j] for j in range(W))
    return y if s["bias"] is None else y + s["bias"]


def _conv(s):
    rows, at, _, tail = _window(s)
    y = _before_silu(s, rows)[at - s["state"].shape[1]]
    if s["silu"]:
        y = y * _sigmoid(y)
    return dict(out=y.to(s["x"].dtype).view(s["x"].shape), state=rows[tail].to(s["x"].dtype))


def _conv_train(s):
    rows, at, head, tail = _window(s)
    io, w, W = s["x"].dtype, s["weight"], s["weight"].shape[1]
    y = _before_silu(s, rows)[at - W + 1]
    d = s["d_out"].reshape(y.shape).float()
    out = y
    if s["silu"]:
        sig = _sigmoid(y)
        out, d = y * sig, d * sig * (1 + y * (1 - sig))
    # zeros behind a sequence's last token: windows of the next one, or what is put behind the rows here
    dy = torch.zeros(len(rows) + W - 1, y.shape[1], device="cuda")
    dy[at] = d
    d_rows = sum(w[:, j] * dy[W - 1 - j:len(dy) - j] for j in range(W))
    d_rows.index_put_((tail,), s["d_state"].float(), accumulate=True)
    d_weight = torch.stack([(d * rows[at - W + 1 + j]).sum(0, dtype=torch.float64) for j in range(W)], 1)
    got = dict(out=out.to(io).view(s["x"].shape), state=rows[tail].to(io), dx=d_rows[at].to(io).view(s["x"].shape), dweight=d_weight.float(), dstate=d_rows[head].to(io))
    if s["bias"] is not None:
        got["dbias"] = d.sum(0, dtype=torch.float64).float()
    return got


def _conv_step(s):
    rows = torch.cat([s["state"].float(), s["x"].float()[:, None]], 1)
    y = (rows * s["weight"].T).sum(1)
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["silu"]:
        y = y * _sigmoid(y)
    s["state"].copy_(rows[:, 1:])
    return dict(out=y.to(s["x"].dtype), state=s["state"])


def _scan(a, x):
    """h_t = a_t h_(t-1) + x_t along the first axis, h_(-1) = 0, by doubling the stretch that each h_t covers."""
    step = 1
    while step < x.shape[0]:
        x = torch.cat([x[:step], x[step:] + a[step:] * x[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return x


def _delta(s):
    """softplus(dt + dt_bias), and its derivative."""
    y = s["dt"].double().reshape(-1, s["dt"].shape[-1]) + s["dt_bias"]
    return torch.clamp(y, min=0) + torch.log1p(torch.exp(-y.abs())), _sigmoid(y)


def _ends(s):
    """First and last row of each sequence that has any, and which sequences these are."""
    cu = _spans(s)
    seq = torch.nonzero(cu[1:] > cu[:-1])[:, 0]
    return cu[seq], cu[seq + 1] - 1, seq


def _states(s):
    """In 64 bits, as states that fade over thousands of tokens multiply as many factors next to 1: the rows' decays, those with none from
    the sequence before, the states, the last ones, delta."""
    delta, _ = _delta(s)
    x, Bm = s["x"].double().flatten(0, 1), s["B"].double().flatten(0, 1)
    a = torch.exp(delta[..., None] * s["A"])
    first, last, seq = _ends(s)
    u = (delta * x)[..., None] * Bm[:, None]
    u.index_put_((first,), a[first] * s["state"][seq].double(), accumulate=True)
    cut = a.index_put((first,), torch.zeros((), dtype=a.dtype, device="cuda"))
    h = _scan(cut, u)
    state = s["state"].clone()
    state[seq] = h[last].float()
    return a, cut, h, state, delta


def _read_out(s, h):
    """(y, silu(z), its derivative)."""
    y = (h * s["C"].double().flatten(0, 1)[:, None]).sum(-1)
    if s["skip"] is not None:
        y = y + s["skip"] * s["x"].flatten(0, 1)
    if s["z"] is None:
        return y, 1.0, None
    z = s["z"].double().flatten(0, 1)
    sig = _sigmoid(z)
    return y, z * sig, sig * (1 + z * (1 - sig))


def _scan_forward(s):
    _, _, h, state, _ = _states(s)
    y, gate, _ = _read_out(s, h)
    return dict(out=(y * gate).to(s["x"].dtype).view(s["x"].shape), state=state)


def _scan_train(s):
    a, cut, h, state, delta = _states(s)
    y, gate, slope = _read_out(s, h)
    io, shape = s["x"].dtype, s["x"].shape
    x, Bm, Cm = (s[n].double().flatten(0, 1) for n in ("x", "B", "C"))
    d_out = s["d_out"].double().flatten(0, 1)
    got = dict(out=(y * gate).to(io).view(shape), state=state)
    if slope is not None:
        got["dz"] = (d_out * y * slope).to(io).view(shape)
    dy = d_out * gate
    first, last, seq = _ends(s)
    d = dy[..., None] * Cm[:, None]
    d.index_put_((last,), s["d_state"][seq].double(), accumulate=True)
    after = torch.cat([cut[1:], torch.zeros_like(cut[:1])])
    dh = _scan(after.flip(0), d.flip(0)).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]]).index_put((first,), s["state"][seq].double())
    got["dC"] = (dy[..., None] * h).sum(1).to(io).view(s["C"].shape)
    got["dB"] = ((delta * x)[..., None] * dh).sum(1).to(io).view(s["B"].shape)
    du = (dh * Bm[:, None]).sum(-1)
    dx = du * delta
    if s["skip"] is not None:
        dx = dx + s["skip"] * dy
        got["dskip"] = (dy * x).sum(0).float()
    got["dx"] = dx.to(io).view(shape)
    got["dstate"] = s["d_state"].clone()
    got["dstate"][seq] = (a[first] * dh[first]).float()
    back = dh * a * before
    got["dA"] = (back * delta[..., None]).sum(0).float()
    d_dt = (du * x + (back * s["A"]).sum(-1)) * _delta(s)[1]
    got["ddt"], got["ddt_bias"] = d_dt.to(io).view(shape), d_dt.sum(0).float()
    return got


def _scan_step(s):
    delta, _ = _delta(s)
    delta = delta.float()
    h = torch.exp(delta[..., None] * s["A"]) * s["state"] + (delta * s["x"].float())[..., None] * s["B"].float()[:, None]
    s["state"].copy_(h)
    y = (h * s["C"].float()[:, None]).sum(-1)
    if s["skip"] is not None:
        y = y + s["skip"] * s["x"].float()
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * _sigmoid(z)
    return dict(out=y.to(s["x"].dtype), state=s["state"])


def _dequantize(codes, scales):
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    x = torch.stack([value[(codes & 15).long()], value[(codes >> 4).long()]], -1).reshape(*codes.shape[:-1], -1, GROUP)
    return torch.ldexp(x, scales[..., None].int() - 127).reshape(*codes.shape[:-1], -1)


def _part(q, keys, values, seen):
    """(largest score, sum of e^(score - largest), weighted values) of queries [n, heads, rows, d] over keys [n, heads, L, d]; seen: [n, rows, L]."""
    scores = torch.matmul(q, keys.transpose(2, 3).contiguous()) / math.sqrt(q.shape[-1])
    scores = scores.masked_fill(~seen[:, None], -math.inf)
    most = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - most)
    return most, p.sum(-1, keepdim=True), torch.matmul(p, values)


def _shared(s):
    """Every group's rows over its prefix, every request's rows over its own tokens, and the two joined."""
    q, cache, table, total, prefix, first = s["q"], s["cache"], s["table"], s["total"].long(), s["prefix"].long(), s["first"].long()
    T, Hq, d = q.shape
    heads, page = cache["k"].shape[1:3]
    share, n = Hq // heads, len(total)
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(n + 1, device="cuda")
    req = torch.searchsorted(cu[1:], torch.arange(T, device="cuda"), right=True)     # of each row
    group = torch.searchsorted(first[1:], torch.arange(n, device="cuda"), right=True)  # of each request

    def gathered(name, rows, at):      # the tokens at positions `at` [m, L] of the tables of `rows` [m]
        page_of = table[rows[:, None], (at // page).clamp(max=table.shape[1] - 1)].clamp(min=0).long()
        x = _dequantize(cache[name][page_of, :, at % page], cache[name + "_scale"][page_of, :, at % page])
        return x.transpose(1, 2).contiguous()

    def part(start, count, table_rows, low, high, most, length):
        """The rows [start, start + count) of q over the tokens from `low` up to `high` (a row's own end where None)."""
        i = torch.arange(most, device="cuda")
        row = (start[:, None] + i).clamp(max=T - 1)                                    # [m, most]
        x = q.float()[row].reshape(len(start), most, heads, share, d).permute(0, 2, 1, 3, 4).reshape(len(start), heads, -1, d)
        at = low[:, None] + torch.arange(length, device="cuda")                       # [m, length]
        end = high[:, None].expand(-1, most) if high is not None else (total[req[row]] - cu[req[row] + 1] + row + 1)
        seen = (at[:, None] < end[..., None]).repeat_interleave(share, 1)
        got = _part(x, gathered("k", table_rows, at), gathered("v", table_rows, at), seen)
        real = i < count[:, None]

        def packed(y):                                                                # [T, Hq, ...]
            return y.view(len(start), heads, most, share, -1).permute(0, 2, 1, 3, 4).reshape(len(start), most, Hq, -1)[real]
        return [packed(y) for y in got]

    heads_of = cu[first]
    m1, s1, o1 = part(heads_of[:-1], heads_of.diff(), first[:-1], torch.zeros_like(prefix), prefix, s["most_rows"], s["most_prefix"])
    m2, s2, o2 = part(cu[:-1], cu.diff(), torch.arange(n, device="cuda"), prefix[group], None, s["most_new"], s["most_own"])
    most = torch.maximum(m1, m2)
    w1, w2 = torch.exp(m1 - most), torch.exp(m2 - most)
    out = (w1 * o1 + w2 * o2) / (w1 * s1 + w2 * s2)
    if s["g"] is not None:
        out = out * _sigmoid(s["g"].float())
    return out.to(q.dtype)


def _own(s):
    import gated_delta_rule_91_amd as kda
    op = s["op"]
    if op == "shared":
        return kda.cache4_shared_attention(s["q"], kda.Cache4(**s["cache"]), s["table"], s["total"], s["prefix"], s["first"], cu_seqlens=s["cu"], g=s["g"],
                                           max_q=s["most_new"], max_prefix=s["most_prefix"], max_own=s["most_own"])
    if op == "conv-step":
        out = kda.short_conv_step(s["x"], s["weight"], s["state"], bias=s["bias"], silu=s["silu"])
        return dict(out=out, state=s["state"])
    if op.startswith("conv"):
        more = dict(bias=s["bias"], silu=s["silu"], state_in=s["state"], cu_seqlens=s["cu"])
        out, state = kda.short_conv_prefill(s["x"], s["weight"], **more)
        got = dict(out=out, state=state)
        if op == "conv-train":
            r = kda.short_conv_backward(s["x"], s["weight"], d_out=s["d_out"], d_state=s["d_state"], **more)
            got.update(dx=r["dx"], dweight=r["dweight"], dstate=r["dstate0"])
            if s["bias"] is not None:
                got["dbias"] = r["dbias"]
        return got
    inputs = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    more = dict(skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"])
    if op == "scan-step":
        out = kda.selective_scan_step(*inputs, s["state"], **more)
        return dict(out=out, state=s["state"])
    more.update(state_in=s["state"], cu_seqlens=s["cu"])
    if op == "scan":
        out, state = kda.selective_scan_prefill(*inputs, **more)
        return dict(out=out, state=state)
    out, state, kept = kda.selective_scan_prefill_for_backward(*inputs, **more)
    r = kda.selective_scan_backward(*inputs, kept, d_out=s["d_out"], d_state=s["d_state"], **more)
    got = dict(out=out, state=state, dstate=r["dstate0"], **{n: r[n] for n in ("dx", "ddt", "dA", "dB", "dC", "ddt_bias")})
    if s["skip"] is not None:
        got["dskip"] = r["dskip"]
    if s["z"] is not None:
        got["dz"] = r["dz"]
    return got


PLAIN = {"conv": _conv, "conv-train": _conv_train, "conv-step": _conv_step, "scan": _scan_forward, "scan-train": _scan_train, "scan-step": _scan_step, "shared": _shared}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------------------

def work(case):
    c = case
    size = DTYPES[c["io"]].itemsize
    if c["op"] == "shared":
        first, prefix, own_lens, new = _shared_lengths(c)
        heads, d = c["kv_heads"], c["d"]
        group = [j for j in range(c["groups"]) for _ in range(first[j], first[j + 1])]
        # each prefix once, every request's own tokens; queries, outputs and gates; tables
        tokens = sum(prefix) + sum(own_lens)
        pairs = sum(m * prefix[j] + m * (2 * o - m + 1) // 2 for j, o, m in zip(group, own_lens, new))
        return dict(bytes=tokens * 2 * heads * (d // 2 + d // GROUP) + sum(new) * c["heads"] * d * size * (3 if c["gate"] else 2) + _pages(tokens, c["page"]) * 4,
                    flops=4 * pairs * c["heads"] * d)
    cells = c["rows"] * c.get("tokens", 1) * c["width"]
    n = c.get("requests") or c["rows"]
    if c["op"].startswith("conv"):
        W = c["taps"]
        params = c["width"] * (W + (1 if c["bias"] else 0)) * 4
        states = n * (W - 1) * c["width"] * size
        if c["op"] == "conv-train":
            # x, d_out read, out, dx written; weights and their gradients; both states and both of their gradients
            return dict(bytes=4 * cells * size + 2 * params + 4 * states, flops=cells * (6 * W + 20))
        return dict(bytes=2 * cells * size + params + 2 * states, flops=cells * (2 * W + 6))
    N, rows = c["states"], c["rows"] * c.get("tokens", 1)
    gate = 1 if c["gate"] else 0
    params, states = c["width"] * (N + 1 + (1 if c["skip"] else 0)) * 4, n * c["width"] * N * 4
    if c["op"] == "scan-train":
        # x, dt, z, d_out read, out, dx, ddt, dz written; B, C and their gradients
        return dict(bytes=cells * size * (6 + 2 * gate) + 4 * rows * N * size + 2 * params + 4 * states, flops=cells * N * 22)
    return dict(bytes=cells * size * (3 + gate) + 2 * rows * N * size + params + 2 * states, flops=cells * N * 7)


# ---- the definitions in 64 bits ---------------------------------------------------------------

def _silu64(x):
    return x * torch.sigmoid(x)


def _exact_conv(c, seed):
    s = prepare(c, seed)
    W, D = c["taps"], c["width"]
    step = c["op"] == "conv-step"
    x = s["x"].double().reshape(-1, D)
    cu = list(range(c["rows"] + 1)) if step else _offsets(c)
    w = s["weight"].double()
    bias = s["bias"].double() if c["bias"] else torch.zeros(D, dtype=torch.float64, device="cuda")
    out, state = torch.empty_like(x), torch.empty(len(cu) - 1, W - 1, D, dtype=torch.float64, device="cuda")
    train = c["op"] == "conv-train"
    if train:
        dx, dw, db, ds = torch.empty_like(x), torch.zeros_like(w), torch.zeros_like(bias), torch.empty_like(state)
        d_out, d_state = s["d_out"].double().reshape(-1, D), s["d_state"].double()
    for r, (b, e) in enumerate(zip(cu, cu[1:])):
        seen = torch.cat([s["state"][r].double(), x[b:e]])
        y = bias.expand(e - b, D).clone()
        for k in range(W):                   # the input k tokens ago
            y += seen[W - 1 - k:W - 1 - k + e - b] * w[:, W - 1 - k]
        out[b:e] = _silu64(y) if c["silu"] else y
        state[r] = seen[e - b:]
        if train:
            d = d_out[b:e]
            if c["silu"]:
                sig = torch.sigmoid(y)
                d = d * (sig + y * sig * (1 - sig))
            back = torch.zeros_like(seen)
            back[e - b:] += d_state[r]
            for k in range(W):
                part = seen[W - 1 - k:W - 1 - k + e - b]
                back[W - 1 - k:W - 1 - k + e - b] += d * w[:, W - 1 - k]
                dw[:, W - 1 - k] += (d * part).sum(0)
            db += d.sum(0)
            dx[b:e], ds[r] = back[W - 1:], back[:W - 1]
    got = dict(out=out.view(s["x"].shape), state=state)
    if train:
        got.update(dx=dx.view(s["x"].shape), dweight=dw, dstate=ds)
        if c["bias"]:
            got["dbias"] = db
    return got


def _exact_scan(c, seed):
    s = prepare(c, seed)
    D, N = c["width"], c["states"]
    step, train = c["op"] == "scan-step", c["op"] == "scan-train"
    n = c.get("requests") or c["rows"]
    if not step and c["requests"]:
        cu = _offsets(c)
        spans = [(slice(0, 1), b, e, slice(r, r + 1)) for r, (b, e) in enumerate(zip(cu, cu[1:]))]
    else:
        spans = [(slice(0, n), 0, 1 if step else c["tokens"], slice(0, n))]     # all rows at once
    x, dt, Bm, Cm = (s[k].double().unsqueeze(1) if step else s[k].double() for k in ("x", "dt", "B", "C"))
    z = None if s["z"] is None else (s["z"].double().unsqueeze(1) if step else s["z"].double())
    raw = dt + s["dt_bias"].double()
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    A = s["A"].double()
    y, state = torch.zeros_like(x), s["state"].double().clone()
    before = torch.zeros(*x.shape, N, dtype=torch.float64, device="cuda") if train else None
    for rows, b, e, at in spans:
        h = state[at].clone()
        for t in range(b, e):
            if train:
                before[rows, t] = h
            h = torch.exp(delta[rows, t, :, None] * A) * h + (delta[rows, t] * x[rows, t])[:, :, None] * Bm[rows, t, None]
            y[rows, t] = (h @ Cm[rows, t, :, None]).squeeze(-1)
        state[at] = h
    if s["skip"] is not None:
        y += s["skip"].double() * x
    out = y if z is None else y * _silu64(z)
    got = dict(out=out.squeeze(1) if step else out, state=state)
    if not train:
        return got
    d_out, ds = s["d_out"].double(), s["d_state"].double().clone()
    dy = d_out if z is None else d_out * _silu64(z)
    dx, dd, dB, dC, dA = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(Bm), torch.zeros_like(Cm), torch.zeros_like(A)
    for rows, b, e, at in spans:
        carry = ds[at].clone()
        for t in range(e - 1, b - 1, -1):
            a = torch.exp(delta[rows, t, :, None] * A)
            u = delta[rows, t] * x[rows, t]
            h = a * before[rows, t] + u[:, :, None] * Bm[rows, t, None]
            dh = carry + dy[rows, t, :, None] * Cm[rows, t, None]
            dC[rows, t] = (dy[rows, t, None] @ h).squeeze(1)
            dB[rows, t] = (u[:, None] @ dh).squeeze(1)
            du = (dh @ Bm[rows, t, :, None]).squeeze(-1)
            carry = a * dh
            back = carry * before[rows, t]
            dx[rows, t] = du * delta[rows, t]
            dd[rows, t] = du * x[rows, t] + (back * A).sum(-1)
            dA += (back * delta[rows, t, :, None]).sum(0)
        ds[at] = carry
    if s["skip"] is not None:
        dx += s["skip"].double() * dy
        got["dskip"] = (dy * x).sum((0, 1))
    ddt = dd * torch.sigmoid(raw)
    got.update(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, ddt_bias=ddt.sum((0, 1)), dstate=ds)
    if z is not None:
        sig = torch.sigmoid(z)
        got["dz"] = d_out * y * (sig + z * sig * (1 - sig))
    return got


def _exact_values(codes, scales):
    half = torch.stack([codes % 16, codes // 16], -1).reshape(*codes.shape[:-1], -1).double()
    size, sign = half % 8, 1 - 2 * (half >= 8).double()
    # 0 and 1/2, then (2 + m) 2^(x - 2) for exponent x and mantissa m
    value = torch.where(size < 2, size / 2, (2 + size % 2) * torch.pow(2.0, torch.floor(size / 2) - 2))
    unit = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=codes.device), scales.double() - 127)
    return sign * value * unit.repeat_interleave(GROUP, -1)


def _exact_shared(c, seed):
    first, prefix, own_lens, new = _shared_lengths(c)
    if sum(new) * c["heads"] * c["prefix"] > 6e9:
        return None
    s = prepare(c, seed)
    page, heads, d = c["page"], c["kv_heads"], c["d"]
    outs, at = [], 0
    for j in range(c["groups"]):
        for r in range(first[j], first[j + 1]):
            t, m = prefix[j] + own_lens[r], new[r]
            whole = torch.arange(t, device="cuda")
            # a request's first tokens are those of the group's first request
            pages = torch.where(whole < prefix[j], s["table"][first[j]][(whole // page).clamp(max=s["table"].shape[1] - 1)], s["table"][r][whole // page]).long()

            def rows(n):
                return _exact_values(s["cache"][n][pages, :, whole % page], s["cache"][n + "_scale"][pages, :, whole % page])

            k, v = rows("k"), rows("v")
            q = s["q"][at:at + m].double()
            hidden = whole > (t - m + torch.arange(m, device="cuda"))[:, None]
            share = c["heads"] // heads
            out = torch.empty_like(q)
            for h in range(heads):
                x = q[:, h * share:(h + 1) * share].reshape(-1, d)
                w = torch.softmax((x @ k[:, h].T / d ** 0.5).masked_fill(hidden.repeat_interleave(share, 0), -math.inf), -1)
                out[:, h * share:(h + 1) * share] = (w @ v[:, h]).view(m, share, d)
            outs.append(out)
            at += m
    out = torch.cat(outs)
    return out * torch.sigmoid(s["g"].double()) if c["gate"] else out


def exact(case, seed):
    if case["op"] == "shared":
        return _exact_shared(case, seed)
    if case["op"].startswith("conv"):
        return _exact_conv(case, seed)
    return _exact_scan(case, seed)
