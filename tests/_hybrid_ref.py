"""Plain 64-bit forms of the operators beside KDA, on the CPU, one token or
one request at a time.  Test infrastructure only."""
import math

import torch

INT32_MAX = 2 ** 31 - 1


def plan(past, new, table, free, page, tokens):
    """(cu, total, slots, table, taken) of lists; the documented bounds included."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    cu, total, slots, taken = [0], [], [], 0
    for r, (p, m) in enumerate(zip(past, new)):
        p, m = max(p, 0), max(m, 0)
        first = min(-(-p // page), width)
        last = min(-(-(p + m) // page), width)
        for j in range(first, last):
            table[r][j] = free[taken] if taken < len(free) else -1
            taken += 1
        for at in range(p, p + min(m, tokens - cu[-1])):
            ok = at // page < width and table[r][at // page] >= 0
            slots.append(table[r][at // page] * page + at % page if ok else -1)
        cu.append(min(cu[-1] + m, tokens))
        total.append(min(p + m, INT32_MAX))
    return cu, total, slots + [-1] * (tokens - len(slots)), table, taken


GRID = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def quantized(x):
    """(codes 0..15 per value, scale byte per 32) of x [..., d], one group at a time."""
    x = x.double()
    flat = x.reshape(-1, 32)
    codes, scales = [], []
    for row in flat.tolist():
        if not all(math.isfinite(v) for v in row):
            codes.append([0] * 32)
            scales.append(255)
            continue
        m = max(abs(v) for v in row)
        e = -125
        if m > 0:
            e = math.frexp(m)[1] - 3
            e += m > 7 * 2.0 ** e
            e = min(max(e, -125), 125)
        out = []
        for v in row:
            y = abs(v) / 2.0 ** e
            k = min(range(8), key=lambda i: (abs(y - GRID[i]), i % 2))   # the nearest, the even one of two
            out.append(k + (8 if math.copysign(1, v) < 0 else 0))
        codes.append(out)
        scales.append(e + 127)
    return (torch.tensor(codes, dtype=torch.uint8).reshape(x.shape),
            torch.tensor(scales, dtype=torch.uint8).reshape(*x.shape[:-1], x.shape[-1] // 32))


def packed(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def values(data, scales):
    """fp64 values of packed codes [..., d/2] and scales [..., d/32]."""
    half = torch.stack([data & 15, data >> 4], -1).flatten(-2)
    grid = torch.tensor(GRID + [-g for g in GRID], dtype=torch.float64)
    unit = torch.pow(torch.tensor(2.0, dtype=torch.float64), scales.double() - 127)
    unit[scales == 255] = math.nan
    return grid[half.long()] * unit.repeat_interleave(32, -1)


def attention(q, cache, table, total, cu, scale, g=None):
    """(out, sum p |v|, bound on the scores' size): cache is a dict of CPU tensors k, k_scale, v, v_scale; rows of no
    sequence are NaN.  Pages outside the cache are left out."""
    T, Hq, d = q.shape
    pages, H, page = cache["k"].shape[:3]
    k = values(cache["k"], cache["k_scale"])
    v = values(cache["v"], cache["v_scale"])
    out = torch.full((T, Hq, d), math.nan, dtype=torch.float64)
    mag, size = torch.zeros_like(out), 0.0
    q = q.double()
    for s in range(len(total)):
        b, e = cu[s], cu[s + 1]
        for row in range(b, e):
            end = total[s] - (e - b) + (row - b) + 1
            seen = [t for t in range(min(end, len(table[s]) * page)) if 0 <= table[s][t // page] < pages]
            at = torch.tensor([table[s][t // page] for t in seen], dtype=torch.long)
            off = torch.tensor([t % page for t in seen], dtype=torch.long)
            for h in range(Hq):
                kv = h // (Hq // H)
                if not seen:
                    out[row, h] = 0
                    continue
                kk, vv = k[at, kv, off], v[at, kv, off]
                w = torch.softmax(kk @ q[row, h] * scale, 0)
                out[row, h] = w @ vv
                mag[row, h] = w @ vv.abs()
                size = max(size, float((kk.abs() @ q[row, h].abs()).max()) * abs(scale))
            if g is not None:
                sig = torch.sigmoid(g[row].double())
                out[row] *= sig
                mag[row] *= sig
    return out, mag, size


def recurrence(x, la, floor, g, state, cu=None, d_out=None, d_state=None):
    """Everything that the recurrence and its backward compute, one token at a time; rows of no sequence are NaN."""
    B, T, D = x.shape
    x, a = x.double(), torch.exp(torch.clamp(torch.nan_to_num(la.double(), nan=-math.inf), min=floor))
    spans = [(r, 0, T, r) for r in range(B)] if cu is None else [(0, cu[s], cu[s + 1], s) for s in range(len(cu) - 1)]
    n = len(spans)
    state = torch.zeros(n, D, dtype=torch.float64) if state is None else state.double()
    sig = torch.sigmoid(g.double()) if g is not None else torch.ones_like(x)
    nan = lambda: torch.full((B, T, D), math.nan, dtype=torch.float64)
    h, before, r = nan(), nan(), {}
    final = torch.zeros(n, D, dtype=torch.float64)
    for row, b, e, s in spans:
        now = state[s]
        for t in range(b, e):
            before[row, t] = now
            now = a[row, t] * now + x[row, t]
            h[row, t] = now
        final[s] = now
    r["out"], r["state"], r["h"] = h * sig, final, h
    if d_out is not None or d_state is not None:
        d_out = torch.zeros_like(x) if d_out is None else d_out.double()
        r["dx"], r["dlog_alpha"], r["dstate0"] = nan(), nan(), torch.zeros(n, D, dtype=torch.float64)
        for row, b, e, s in spans:
            carry = torch.zeros(D, dtype=torch.float64) if d_state is None else d_state[s].double()
            for t in range(e - 1, b - 1, -1):
                dh = d_out[row, t] * sig[row, t] + carry
                carry = a[row, t] * dh
                r["dx"][row, t] = dh
                r["dlog_alpha"][row, t] = torch.where(la[row, t].double() > floor, carry * before[row, t], 0.0)
            r["dstate0"][s] = carry
        r["dg"] = d_out * h * sig * (1 - sig)
    return r
