"""Plain 64-bit forms of the short convolution and the selective scan, on the
CPU, one sequence and one token at a time, with bounds on how far a form in 32
bits may be off.  Test infrastructure only.

The bounds are first-order running error bounds: beside every value goes what the
roundings of its parts can add up to, u = 2^-24 each.  They leave out the rounding
of a stored result to its own type, which the tests add."""
import torch

U = 2.0 ** -24
LEAST = 2.0 ** -126


def _sig(x):
    return torch.sigmoid(x)


def _spans(rows, T, cu):
    """(row, first, end, sequence) of every sequence."""
    if cu is None:
        return [(r, 0, T, r) for r in range(rows)]
    return [(0, cu[s], cu[s + 1], s) for s in range(len(cu) - 1)]


def conv(x, weight, bias, silu, state, cu=None, d_out=None, d_state=None):
    """{name: (value, bound)}; rows of no sequence are NaN.

    A sum of W products and a bias: (W + 1) u of the sum of their sizes.  sigmoid
    has its argument's rounding (2 |y| u), an exponential, a sum and a reciprocal
    (12 u); silu' = s (1 + y (1 - s)) multiplies that by 1 + |y|, twice where 1 - s
    is next to 0.  A weight's gradient adds up a tile of 64 tokens in 32 bits."""
    B, T, D = x.shape
    W = weight.shape[1]
    x, w = x.double(), weight.double()
    b = torch.zeros(D, dtype=torch.float64) if bias is None else bias.double()
    spans = _spans(B, T, cu)
    n = len(spans)
    state = torch.zeros(n, W - 1, D, dtype=torch.float64) if state is None else state.double()
    nan = lambda: torch.full((B, T, D), float("nan"), dtype=torch.float64)
    out, e_out, dx, e_dx = nan(), nan(), nan(), nan()
    last, ds, e_ds = torch.zeros_like(state), torch.zeros_like(state), torch.zeros_like(state)
    dw, e_dw, db, e_db = torch.zeros_like(w), torch.zeros_like(w), torch.zeros_like(b), torch.zeros_like(b)
    back = d_out is not None or d_state is not None
    for row, first, end, s in spans:
        m = end - first
        seen = torch.cat([state[s], x[row, first:end]])
        parts = torch.stack([seen[j:j + m] * w[:, j] for j in range(W)])
        y = parts.sum(0) + b
        ey = (W + 1) * U * (parts.abs().sum(0) + b.abs())
        sig = _sig(y)
        out[row, first:end] = y * sig if silu else y
        e_out[row, first:end] = 1.1 * ey + (2 * y.abs() + 16) * U * (y * sig).abs() if silu else ey
        last[s] = seen[m:]
        if not back:
            continue
        d = torch.zeros_like(y) if d_out is None else d_out[row, first:end].double()
        ed = torch.zeros_like(d)
        if silu:
            ed = d.abs() * (0.5 * ey + (8 * y.abs() + 32) * (1 + y.abs()) * U * sig)
            d = d * sig * (1 + y * (1 - sig))
        g, eg = torch.zeros_like(seen), torch.zeros_like(seen)
        if d_state is not None:
            g[m:] += d_state[s].double()
            eg[m:] += U * d_state[s].double().abs()
        for j in range(W):
            g[j:j + m] += d * w[:, j]
            eg[j:j + m] += ed * w[:, j].abs() + (W + 2) * U * (d * w[:, j]).abs()
            dw[:, j] += (d * seen[j:j + m]).sum(0)
            e_dw[:, j] += ((ed + 72 * U * d.abs()) * seen[j:j + m].abs()).sum(0)
        db += d.sum(0)
        e_db += (ed + 72 * U * d.abs()).sum(0)
        dx[row, first:end], e_dx[row, first:end] = g[W - 1:], eg[W - 1:]
        ds[s], e_ds[s] = g[:W - 1], eg[:W - 1]
    r = dict(out=(out, e_out), state=(last, torch.zeros_like(last)))
    if back:
        r.update(dx=(dx, e_dx), dweight=(dw, e_dw), dbias=(db, e_db), dstate0=(ds, e_ds))
    return r


def scan(x, dt, A, B, C, skip=None, z=None, dt_bias=None, state=None, cu=None, d_out=None, d_state=None, tile=64):
    """{name: (value, bound)}; rows of no sequence are NaN.

    delta is off by (|dt + bias| + 12) u of itself (the sum's rounding, an
    exponential, a quotient and a series); a decay by (delta |A|) times what its
    exponent is off (4 u more) and 3 u, and one below 2^-126, the least normal
    number, may count as 0; a step rounds twice.  Where tiles are joined, sums of
    up to `tile` deltas round as often, which shifts a term by at most
    max(l e^-l) = 0.37 times that, and decays over several tokens may underflow
    too.  Sums over states take N u of their sizes,
    sums over channels D u, sums over a tile's tokens tile u.  Gates as in conv."""
    R, T, D = x.shape
    N = A.shape[1]
    x, dt, A, B, C = (t.double() for t in (x, dt, A, B, C))
    zero = torch.zeros(D, dtype=torch.float64)
    skip_, bias = (zero if t is None else t.double() for t in (skip, dt_bias))
    spans = _spans(R, T, cu)
    n = len(spans)
    state = torch.zeros(n, D, N, dtype=torch.float64) if state is None else state.double()
    raw = dt + bias
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    rd = (raw.abs() + 12) * U                       # relative, of delta
    sz = None if z is None else _sig(z.double())
    gate = torch.ones_like(x) if z is None else z.double() * sz
    rg = torch.zeros_like(x) if z is None else (2 * z.double().abs() + 16) * U
    nan = lambda *shape: torch.full(shape, float("nan"), dtype=torch.float64)
    y, ey, final, e_final = nan(R, T, D), nan(R, T, D), torch.zeros_like(state), torch.zeros_like(state)
    back = d_out is not None or d_state is not None
    hs, ehs, befores, e_befores = {}, {}, {}, {}
    absA = A.abs()

    def decay(row, t):
        lam = delta[row, t, :, None] * absA
        a = torch.exp(delta[row, t, :, None] * A)
        return a, lam * (rd[row, t, :, None] + 4 * U) + 3 * U + LEAST / a.clamp(min=1e-300)

    def joined(size, total):
        return 0.37 * tile * U * size + LEAST * total

    for row, first, end, s in spans:
        h, eh, size, total = state[s].clone(), torch.zeros_like(state[s]), state[s].abs(), state[s].abs()
        for t in range(first, end):
            a, ra = decay(row, t)
            if back:
                befores[row, t], e_befores[row, t] = h, eh + joined(size, total)
            u = (delta[row, t] * x[row, t])[:, None] * B[row, t]
            eh = a * eh + (a * h).abs() * ra + u.abs() * (rd[row, t, :, None] + 3 * U)
            size, total = a * size + u.abs(), total + u.abs()
            h = a * h + u
            eh = eh + 2 * U * h.abs()
            e = eh + joined(size, total)
            if back:
                hs[row, t], ehs[row, t] = h, e
            terms = h * C[row, t]
            y[row, t] = terms.sum(-1) + skip_ * x[row, t]
            ey[row, t] = (e * C[row, t].abs()).sum(-1) + (N + 4) * U * (terms.abs().sum(-1) + (skip_ * x[row, t]).abs())
        final[s], e_final[s] = h, eh + joined(size, total)
    r = dict(out=(y * gate, ey * gate.abs() + (y * gate).abs() * (rg + 2 * U)), state=(final, e_final))
    if not back:
        return r
    d_out = torch.zeros_like(x) if d_out is None else d_out.double()
    dy, edy = d_out * gate, (d_out * gate).abs() * (rg + U)
    if z is not None:
        zz = z.double()
        slope = sz * (1 + zz * (1 - sz))
        r["dz"] = (d_out * y * slope, (d_out * slope).abs() * ey + (d_out * y).abs() * ((8 * zz.abs() + 32) * (1 + zz.abs()) * U * sz + 4 * U * slope.abs()))
    dx, e_dx, dd, e_dd = nan(R, T, D), nan(R, T, D), nan(R, T, D), nan(R, T, D)
    dB, e_dB, dC, e_dC = (nan(R, T, N) for _ in range(4))
    dA, e_dA, ds, e_ds = (torch.zeros(*sh, dtype=torch.float64) for sh in ((D, N), (D, N), (n, D, N), (n, D, N)))
    for row, first, end, s in spans:
        g = torch.zeros_like(state[s]) if d_state is None else d_state[s].double()
        eg, size, total = torch.zeros_like(g), g.abs(), g.abs()
        for t in range(end - 1, first - 1, -1):
            a, ra = decay(row, t)
            c, e_c = C[row, t] * dy[row, t, :, None], C[row, t].abs() * (edy[row, t, :, None] + 2 * U * dy[row, t, :, None].abs())
            dh, e_dh = c + g, e_c + eg + joined(size, total) + U * (c.abs() + g.abs())
            w = delta[row, t] * x[row, t]
            dC[row, t] = (dy[row, t, :, None] * hs[row, t]).sum(0)
            e_dC[row, t] = (dy[row, t, :, None].abs() * ehs[row, t] + (edy[row, t, :, None] + (D + 4) * U * dy[row, t, :, None].abs()) * hs[row, t].abs()).sum(0)
            dB[row, t] = (w[:, None] * dh).sum(0)
            e_dB[row, t] = (w[:, None].abs() * (e_dh + (rd[row, t, :, None] + (D + 4) * U) * dh.abs())).sum(0)
            terms = dh * B[row, t]
            du, e_du = terms.sum(-1), (e_dh * B[row, t].abs()).sum(-1) + (N + 2) * U * terms.abs().sum(-1)
            back_ = a * dh * befores[row, t]
            e_b = a * (e_dh * befores[row, t].abs() + dh.abs() * e_befores[row, t]) + back_.abs() * (ra + 4 * U)
            dx[row, t] = du * delta[row, t] + skip_ * dy[row, t]
            e_dx[row, t] = e_du * delta[row, t] + (du * delta[row, t]).abs() * (rd[row, t] + 3 * U) + skip_.abs() * (edy[row, t] + 3 * U * dy[row, t].abs())
            dd[row, t] = du * x[row, t] + (back_ * A).sum(-1)
            e_dd[row, t] = (e_du + 3 * U * du.abs()) * x[row, t].abs() + ((e_b + (N + 6) * U * back_.abs()) * absA).sum(-1)
            dA += back_ * delta[row, t, :, None]
            e_dA += (e_b + (rd[row, t, :, None] + (tile + 4) * U) * back_.abs()) * delta[row, t, :, None]
            eg = a * (e_c + eg + U * (c.abs() + g.abs())) + (a * dh).abs() * (ra + U)
            size, total = a * (size + c.abs()), total + c.abs()
            g = a * dh
        ds[s], e_ds[s] = g, eg + joined(size, total)
    sig = _sig(raw)
    ddt = dd * sig
    e_ddt = (e_dd + dd.abs() * (2 * raw.abs() + 16) * U) * sig
    r.update(dx=(dx, e_dx), ddt=(ddt, e_ddt), dA=(dA, e_dA), dB=(dB, e_dB), dC=(dC, e_dC), dstate0=(ds, e_ds))
    live = ~torch.isnan(dx)
    overall = lambda v: torch.where(live, v, 0.0).sum((0, 1))
    r["dskip"] = (overall(dy * x), overall((edy + (tile + 4) * U * dy.abs()) * x.abs()))
    r["ddt_bias"] = (overall(ddt), overall(e_ddt + (tile + 4) * U * ddt.abs()))
    return r
