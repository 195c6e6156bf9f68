"""The gated linear recurrence on an MI355X against a plain 64-bit form.

Tolerance, from the roundings that the kernel may make.  A step rounds twice
(2 u, u = 2^-24), expm1 is off by 4 u of itself, and each rounding fades as the
state does: a channel that remembers N tokens (1 / (1 - a), at most T) sums
(2 N + 8) of them, and joining tiles adds a few a tile, below one a token.  So
states are within (3 N + 16) u max |h|, and in reverse dh within (3 N + 16) u
max |dh|; products add the errors of their factors; a gate is off by 8 u; an
output rounds once, u of its type."""
import math

import pytest

import _hybrid_ref as ref

torch = pytest.importorskip("torch")
import gated_delta_rule_91_amd as kda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
UO = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24
FLOOR = -0.5


def made(B, T, D, io, n=None, gate=True, seed=0, slowest=-7.0):
    gen = torch.Generator(device="cuda").manual_seed(seed + B * 7 + T * 3 + D)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    slow = torch.rand(D, generator=gen, device="cuda") * (slowest - 1) + 1     # up to e: beyond the floor
    la = -torch.exp(slow + 0.3 * r(B, T, D))
    x, g, d_out = (r(B, T, D).to(DT[io]) for _ in range(3))
    n = B if n is None else n
    return dict(x=x, la=la, g=g if gate else None, s0=r(n, D), d_out=d_out, d_state=r(n, D))


def bounds(i, want, io):
    """Per channel tolerances of h and dh, from the documented rule."""
    T = i["x"].shape[1]
    least = -torch.clamp(torch.nan_to_num(i["la"].double(), nan=-math.inf), min=FLOOR).cpu()
    mem = torch.clamp(1 / torch.clamp(1 - torch.exp(-least.amin((0, 1))), min=1e-9), max=T) if T else torch.zeros(least.shape[-1])
    return (3 * mem + 16) * U


def within(got, want, tol, label):
    got, want = got.cpu().double(), want
    keep = ~torch.isnan(want)
    worst = ((got - want).abs() / (tol + 1e-30))[keep]
    assert worst.numel() == 0 or float(worst.max()) <= 1, (label, float(worst.max()))


def check(i, io, cu=None, backward=True):
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    cpu = {k: None if v is None else v.cpu() for k, v in i.items()}
    want = ref.recurrence(cpu["x"], cpu["la"], FLOOR, cpu["g"], cpu["s0"], cu, cpu["d_out"], cpu["d_state"])
    k = bounds(i, want, io)
    top = lambda x: torch.nan_to_num(x).abs().flatten(0, -2).amax(0) if x.numel() else torch.zeros(x.shape[-1], dtype=torch.float64)
    s0 = torch.zeros(1, i["x"].shape[2], dtype=torch.float64) if cpu["s0"] is None else cpu["s0"].double()
    th = k * torch.maximum(top(want["h"]), top(s0))
    room = torch.full((i["x"].numel() + 64,), 55.0, dtype=i["x"].dtype, device="cuda")
    out = room[:i["x"].numel()].view(i["x"].shape)        # nothing is written behind it
    got, state = kda.recurrence_prefill(i["x"], i["la"], FLOOR, g=i["g"], state_in=i["s0"], cu_seqlens=cut, out=out)
    torch.cuda.synchronize()
    assert (room[i["x"].numel():] == 55.0).all()
    left = torch.isnan(want["out"])
    assert (out.cpu()[left] == 55.0).all()                # tokens of no sequence
    within(out, want["out"], th + 8 * U * want["out"].abs() + UO[io] * want["out"].abs(), "out")
    within(state, want["state"], th, "state")
    if not backward:
        return
    out2, state2, ws = kda.recurrence_prefill_for_backward(i["x"], i["la"], FLOOR, g=i["g"], state_in=i["s0"], cu_seqlens=cut)
    torch.cuda.synchronize()
    assert torch.equal(out2.cpu()[~left], out.cpu()[~left]) and torch.equal(state2, state)
    ds = torch.zeros_like(s0) if cpu["d_state"] is None else cpu["d_state"].double()
    td = k * torch.maximum(top(want["dx"]), top(ds))
    a = torch.exp(torch.clamp(torch.nan_to_num(cpu["la"].double(), nan=-math.inf), min=FLOOR))
    before = torch.maximum(top(want["h"]), top(s0))
    for _ in range(2):                                    # the workspace serves a second call
        r = kda.recurrence_backward(i["x"], i["la"], FLOOR, ws, g=i["g"], state_in=i["s0"], cu_seqlens=cut,
                                    d_out=i["d_out"], d_state=i["d_state"])
        torch.cuda.synchronize()
        within(r["dx"], want["dx"], td + UO[io] * want["dx"].abs(), "dx")
        tl = a * (td * before + th * torch.maximum(top(want["dx"]), top(ds))) + 16 * U * want["dlog_alpha"].abs()
        within(r["dlog_alpha"], want["dlog_alpha"], tl, "dlog_alpha")
        within(r["dstate0"], want["dstate0"], td, "dstate0")
        if i["g"] is not None:
            d = torch.zeros_like(want["h"]) if cpu["d_out"] is None else cpu["d_out"].double()
            # sigmoid and 1 - sigmoid are off by 4 u of 1 each
            within(r["dg"], want["dg"], d.abs() * (th + 16 * U * want["h"].abs()) + UO[io] * want["dg"].abs(), "dg")
        else:
            assert r["dg"] is None


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (2, 63, 5), (3, 64, 64), (1, 65, 129), (2, 255, 66), (1, 256, 128), (1, 257, 130),
                                   (2, 1000, 34), (1, 2500, 257), (5, 7, 300)])
def test_uniform(B, T, D, gate, io):
    check(made(B, T, D, io, gate=gate), io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("cu,T,D", [([0, 5], 5, 3), ([0, 1, 2, 3], 3, 64), ([0, 64, 128], 128, 130), ([0, 0, 70, 70, 70, 300, 300], 300, 66),
                                    ([0, 255, 256, 257, 513, 1400], 1400, 33), ([3, 10, 200], 260, 128),
                                    ([0, 1300], 1300, 200), ([0, 0], 40, 8), ([2, 600, 600, 1025], 1030, 65)])
def test_packed(cu, T, D, io):
    check(made(1, T, D, io, n=len(cu) - 1), io, cu=cu)


def test_packed_many_short_sequences():
    gen = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 9, (400,), generator=gen).tolist()
    cu = [0]
    for m in lens:
        cu.append(cu[-1] + m)
    check(made(1, cu[-1], 70, "f32", n=400), "f32", cu=cu)


def test_packed_equals_alone():
    """A sequence gives the same in a batch as alone, to the tolerance of both (their tiles lie otherwise)."""
    cu = [0, 300, 1100]
    i = made(1, 1100, 64, "f32", n=2)
    check(i, "f32", cu=cu)
    for s in range(2):
        j = {k: v[:, cu[s]:cu[s + 1]].contiguous() if v.dim() == 3 else v[s:s + 1].contiguous() for k, v in i.items()}
        check(j, "f32")


@pytest.mark.parametrize("B,T,D", [(1, 4000, 64), (2, 700, 31)])
def test_slow_channels(B, T, D):
    """Channels that remember thousands of tokens."""
    check(made(B, T, D, "f32", slowest=-10.0), "f32")


def test_optional_arguments():
    for name in ("s0", "d_out", "d_state"):
        i = made(2, 300, 40, "f32")
        i[name] = None
        check(i, "f32")
    i = made(2, 300, 40, "f32")
    out, state = kda.recurrence_prefill(i["x"], i["la"], FLOOR, want_state=False)
    assert state is None
    _, _, ws = kda.recurrence_prefill_for_backward(i["x"], i["la"], FLOOR)
    assert kda.recurrence_backward(i["x"], i["la"], FLOOR, ws, d_out=i["d_out"], want_dstate=False)["dstate0"] is None


def test_no_tokens():
    z = lambda *s: torch.zeros(*s, device="cuda")
    s0 = torch.randn(3, 20, device="cuda")
    for x, cu in ((z(3, 0, 20), None), (z(1, 0, 20), torch.zeros(4, dtype=torch.int32, device="cuda"))):
        out, state, ws = kda.recurrence_prefill_for_backward(x, x, FLOOR, state_in=s0, cu_seqlens=cu)
        r = kda.recurrence_backward(x, x, FLOOR, ws, state_in=s0, cu_seqlens=cu, d_state=2 * s0)
        torch.cuda.synchronize()
        assert torch.equal(state, s0) and torch.equal(r["dstate0"], 2 * s0)
    out, state = kda.recurrence_prefill(z(0, 5, 20), z(0, 5, 20), FLOOR)
    assert out.shape == (0, 5, 20) and state.shape == (0, 20)
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, state = kda.recurrence_prefill(z(1, 5, 20), z(1, 5, 20), FLOOR, cu_seqlens=none, out=torch.full((1, 5, 20), 9.0, device="cuda"))
    torch.cuda.synchronize()
    assert (out == 9).all() and state.shape == (0, 20)


def test_floor_nan_and_infinities():
    i = made(1, 600, 16, "f32")
    i["la"][0, 10, 0] = math.nan                          # acts as the floor
    i["la"][0, 300, 1] = -math.inf
    i["la"][0, :, 2] = FLOOR                              # the floor binds: no gradient
    check(i, "f32")
    x, la = i["x"].clone(), i["la"]
    x[0, 100, 3] = math.nan                               # stays in its channel, from its token on
    x[0, 270, 4] = math.inf
    out, state = kda.recurrence_prefill(x, la, FLOOR, state_in=i["s0"])
    torch.cuda.synchronize()
    bad = ~torch.isfinite(out.cpu()[0])
    want = torch.zeros_like(bad)
    want[100:, 3] = True
    want[270:, 4] = True
    assert torch.equal(bad, want)
    # no floor: a decay to nothing forgets
    la = la.clone()
    la[0, 50] = -math.inf
    out, state = kda.recurrence_prefill(i["x"], la, -math.inf)
    torch.cuda.synchronize()
    assert torch.equal(out[0, 50], i["x"][0, 50])


def test_state_in_place():
    for B, T in ((3, 40), (2, 900)):
        i = made(B, T, 50, "f32")
        out, state = kda.recurrence_prefill(i["x"], i["la"], FLOOR, state_in=i["s0"])
        s = i["s0"].clone()
        out2, same = kda.recurrence_prefill(i["x"], i["la"], FLOOR, state_in=s, state_out=s)
        torch.cuda.synchronize()
        assert same is s and torch.equal(s, state) and torch.equal(out, out2)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 2, 3, 127])
def test_narrow_and_long(D, io):
    """The chain of tiles alone: widths below, at and around a pair of channels."""
    check(made(2, 1500, D, io), io)
    cu = [0, 130, 130, 131, 900, 1500]
    check(made(1, 1500, D, io, n=5), io, cu=cu)


def test_same_bits_every_time():
    i = made(1, 6000, 514, "bf16")
    first = None
    for _ in range(6):
        out, state, ws = kda.recurrence_prefill_for_backward(i["x"], i["la"], FLOOR, g=i["g"], state_in=i["s0"])
        r = kda.recurrence_backward(i["x"], i["la"], FLOOR, ws, g=i["g"], state_in=i["s0"], d_out=i["d_out"], d_state=i["d_state"])
        torch.cuda.synchronize()
        now = [out, state] + [r[k] for k in ("dx", "dlog_alpha", "dg", "dstate0")]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(now, first))


@pytest.mark.parametrize("B,T,D", [(64, 40, 129), (3, 700, 129), (2, 300, 257), (5, 130, 127), (4, 200, 3)])
def test_state_in_place_of_odd_widths(B, T, D):
    """A channel that two lanes share: neither reads a state that the other has written."""
    i = made(B, T, D, "bf16")
    out, state = kda.recurrence_prefill(i["x"], i["la"], FLOOR, g=i["g"], state_in=i["s0"])
    s = i["s0"].clone()
    out2, same = kda.recurrence_prefill(i["x"], i["la"], FLOOR, g=i["g"], state_in=s, state_out=s)
    torch.cuda.synchronize()
    assert same is s and torch.equal(s, state) and torch.equal(out, out2)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N,D", [(1, 1), (3, 77), (7, 128), (300, 96)])
def test_step(N, D, io):
    i = made(N, 1, D, io)
    want = ref.recurrence(i["x"].cpu(), i["la"].cpu(), FLOOR, i["g"].cpu(), i["s0"].cpu())
    state = i["s0"].clone()
    out = kda.recurrence_step(i["x"][:, 0].contiguous(), i["la"][:, 0].contiguous(), state, FLOOR, g=i["g"][:, 0].contiguous())
    torch.cuda.synchronize()
    size = want["h"][:, 0].abs() + i["s0"].cpu().double().abs() + i["x"].cpu().double()[:, 0].abs()
    within(state, want["state"], 8 * U * size, "state")
    within(out, want["out"][:, 0], 16 * U * size + UO[io] * want["out"][:, 0].abs(), "out")


def test_gradients_against_differences():
    """Central differences of the 64-bit form, for a few entries of every input."""
    i = made(1, 300, 6, "f32", n=2)
    cu = [0, 120, 300]
    leaves = {k: i[k].clone().requires_grad_(True) for k in ("x", "la", "g", "s0")}
    out, state = kda.recurrence_autograd(leaves["x"], leaves["la"], FLOOR, g=leaves["g"], state_in=leaves["s0"],
                                         cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    ((out * i["d_out"]).sum() + (state * i["d_state"]).sum()).backward()
    torch.cuda.synchronize()
    cpu = {k: v.cpu().double() for k, v in i.items()}

    def loss(**kw):
        a = {**cpu, **kw}
        r = ref.recurrence(a["x"], a["la"], FLOOR, a["g"], a["s0"], cu)
        return float((r["out"] * cpu["d_out"]).sum() + (r["state"] * cpu["d_state"]).sum())

    eps = 1e-5
    for k, leaf in leaves.items():
        for at in ((0, 0, 1), (0, 119, 2), (0, 120, 3), (0, 257, 4)) if leaf.dim() == 3 else ((0, 2), (1, 5)):
            if k == "la" and abs(float(cpu[k][at]) - FLOOR) < 1e-3:
                continue
            up, down = cpu[k].clone(), cpu[k].clone()
            up[at] += eps
            down[at] -= eps
            diff = (loss(**{k: up}) - loss(**{k: down})) / (2 * eps)
            # differences of second order: eps^2 times third derivatives, and 1e-11 of the loss's rounding over eps
            assert abs(float(leaf.grad[at]) - diff) <= 1e-4 * max(1.0, abs(diff)), (k, at)


def test_given_workspaces():
    """Whatever a workspace holds before; too small a one is refused."""
    i = made(2, 700, 34, "f32")
    p = kda.recurrence_problem(2, 700, 34, torch.float32, FLOOR)
    sizes = kda.recurrence_workspace_size(p), kda.recurrence_backward_workspace_size(p)
    assert sizes[1] > sizes[0] > 0
    want, state, ws = kda.recurrence_prefill_for_backward(i["x"], i["la"], FLOOR, g=i["g"], state_in=i["s0"])
    grads = kda.recurrence_backward(i["x"], i["la"], FLOOR, ws, g=i["g"], state_in=i["s0"], d_out=i["d_out"])
    for fill in (0, 255, 128):
        ws = [torch.full((n,), fill, dtype=torch.uint8, device="cuda") for n in sizes]
        for _ in range(2):
            out, s1 = kda.recurrence_prefill(i["x"], i["la"], FLOOR, g=i["g"], state_in=i["s0"], workspace=ws[0])
            out2, s2, _ = kda.recurrence_prefill_for_backward(i["x"], i["la"], FLOOR, g=i["g"], state_in=i["s0"], workspace=ws[1])
            r = kda.recurrence_backward(i["x"], i["la"], FLOOR, ws[1], g=i["g"], state_in=i["s0"], d_out=i["d_out"])
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(out2, want) and torch.equal(s1, state) and torch.equal(s2, state)
            assert all(torch.equal(r[k], grads[k]) for k in r)
    for call in (lambda: kda.recurrence_prefill(i["x"], i["la"], FLOOR, workspace=ws[0][:-256]),
                 lambda: kda.recurrence_prefill_for_backward(i["x"], i["la"], FLOOR, workspace=ws[1][:-256]),
                 lambda: kda.recurrence_backward(i["x"], i["la"], FLOOR, ws[1][:-256], d_out=i["d_out"])):
        with pytest.raises(kda.KdaError) as e:
            call()
        assert e.value.code == 3


def test_offsets_past_32_bits():
    """Over 2^31 elements: the last of the rows is what it is alone."""
    B, T, D = 3, 175000, 4100
    x = torch.zeros(B, T, D, dtype=torch.bfloat16, device="cuda")
    la = torch.full((B, T, D), -0.01, device="cuda")
    assert x.numel() > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(9)
    x[2, -500:] = torch.randn(500, D, generator=gen, device="cuda").bfloat16()
    la[2, -300:] = -torch.rand(300, D, generator=gen, device="cuda")
    out, state = kda.recurrence_prefill(x, la, FLOOR)
    torch.cuda.synchronize()
    assert not out[0].any() and not out[1].any() and not out[2, :-500].any()
    ref_out, ref_state = kda.recurrence_prefill(x[2:, -500:].contiguous(), la[2:, -500:].contiguous(), FLOOR)
    torch.cuda.synchronize()
    # both are within (3 N + 16) u of the formula, N <= 100 here, and round once more
    top = float(ref_state.abs().max()) * 2 + 10
    assert torch.allclose(state[2:], ref_state, rtol=0, atol=2 * (3 * 100 + 16) * U * top)
    assert torch.allclose(out[2:, -500:].float(), ref_out.float(), rtol=2 * UO["bf16"], atol=2 * (3 * 100 + 16) * U * top)
    del x, la, out
    torch.cuda.empty_cache()


def test_autograd_refuses_second_derivatives():
    x = torch.randn(1, 20, 4, device="cuda", requires_grad=True)
    out, _ = kda.recurrence_autograd(x, -torch.rand(1, 20, 4, device="cuda"), FLOOR)
    grad, = torch.autograd.grad(out.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        grad.sum().backward()


def test_autograd_of_outputs_that_are_not_used():
    i = made(2, 100, 10, "bf16")
    x = i["x"].clone().requires_grad_(True)
    out, state = kda.recurrence_autograd(x, i["la"], FLOOR)
    state.sum().backward()
    _, _, ws = kda.recurrence_prefill_for_backward(i["x"], i["la"], FLOOR)
    r = kda.recurrence_backward(i["x"], i["la"], FLOOR, ws, d_state=torch.ones(2, 10, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(x.grad, r["dx"])


@pytest.mark.parametrize("D", [5, 515])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_autograd_of_outputs_that_are_joined(D, io):
    """The gradients of a concatenation are views of one array, wherever they begin: the second's is at an odd place."""
    parts = [made(1, T, D, io, seed=T) for T in (3, 70, 9)]

    def leaves(i):
        return [i[k].clone().requires_grad_(True) for k in ("x", "la", "g", "s0")]

    def go(l):
        return kda.recurrence_autograd(l[0], l[1], FLOOR, g=l[2], state_in=l[3])

    joined, alone = [leaves(i) for i in parts], [leaves(i) for i in parts]
    outs = [go(l) for l in joined]
    d_out = torch.cat([i["d_out"] for i in parts], 1)
    d_state = torch.cat([i["d_state"] for i in parts], 1)
    torch.autograd.backward([torch.cat([o for o, _ in outs], 1), torch.cat([s for _, s in outs], 1)], [d_out, d_state])
    for l, i in zip(alone, parts):
        torch.autograd.backward(list(go(l)), [i["d_out"], i["d_state"]])
    torch.cuda.synchronize()
    for a, b in zip(joined, alone):
        assert all(torch.equal(x.grad, y.grad) for x, y in zip(a, b))


@pytest.mark.parametrize("cu,T", [([0, 90, 300], 420), ([7, 7, 60], 61), ([0, 0], 150)])
def test_autograd_of_a_padded_batch(cu, T):
    """Tokens of no sequence: zeros come out and go back, whatever their inputs and what the memory held."""
    i = made(1, T, 66, "bf16", n=len(cu) - 1)
    outside = torch.ones(T, dtype=torch.bool)
    outside[cu[0]:cu[-1]] = False
    for k in ("x", "la", "g"):
        i[k][:, outside.cuda()] = math.nan
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    leaves = [i[k].clone().requires_grad_(True) for k in ("x", "la", "g", "s0")]
    junk = [torch.full_like(i[k], math.nan) for k in ("x", "la", "x", "la", "x", "x") for _ in range(3)]
    torch.cuda.synchronize()
    del junk                                              # what the outputs' memory holds
    out, state = kda.recurrence_autograd(leaves[0], leaves[1], FLOOR, g=leaves[2], state_in=leaves[3], cu_seqlens=cut)
    torch.autograd.backward([out, state], [i["d_out"], i["d_state"]])
    torch.cuda.synchronize()
    for t in (out, *(l.grad for l in leaves[:3])):
        assert not t[0, outside.cuda()].any()
    o, s, ws = kda.recurrence_prefill_for_backward(i["x"], i["la"], FLOOR, g=i["g"], state_in=i["s0"], cu_seqlens=cut)
    r = kda.recurrence_backward(i["x"], i["la"], FLOOR, ws, g=i["g"], state_in=i["s0"], cu_seqlens=cut, d_out=i["d_out"],
                                d_state=i["d_state"])
    torch.cuda.synchronize()
    inside = ~outside.cuda()
    assert torch.equal(state, s) and torch.equal(leaves[3].grad, r["dstate0"])
    for a, b in zip((out, *(l.grad for l in leaves[:3])), (o, r["dx"], r["dlog_alpha"], r["dg"])):
        assert torch.equal(a[0, inside], b[0, inside])


def same_where_not_finite(got, want, label):
    """Inf where the 64-bit form has Inf, of the same sign, and NaN where it has NaN."""
    got = got.detach().cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), label
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf]), label


# decays of a channel: none, slow ones on both sides of 1/16, fast ones, ones that vanish in 32 bits, mixed, and a reset
INF_DECAYS = [0.0, -1e-9, -0.001, -0.0625, -0.0626, -0.4, -3.0, -30.0, -95.0, -300.0, None, "reset"]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,at", [(9, 4), (300, 130), (700, 3)])
def test_infinite_states_stay_infinite(T, at, io):
    D = len(INF_DECAYS)
    i = made(2, T, D, io, gate=False)
    for c, l in enumerate(INF_DECAYS):
        if l is None:
            i["la"][:, ::3, c], i["la"][:, 1::3, c] = -0.02, -2.0
        elif l == "reset":
            i["la"][:, at + 2, c] = -math.inf            # nothing of it is left, which for Inf is NaN
        else:
            i["la"][:, :, c] = l
    i["s0"][1] = -math.inf
    x, d = i["x"].clone(), i["d_out"].clone()
    x[0, at], d[:, -3], d[1, 1] = math.inf, -math.inf, -math.inf
    run = lambda x, d_out: ref.recurrence(x.cpu(), i["la"].cpu(), -math.inf, None, i["s0"].cpu(), None, d_out.cpu(), i["d_state"].cpu())
    want = run(x, i["d_out"])
    assert torch.isinf(want["out"][0, at:, :-1]).all() and torch.isnan(want["out"][0, at + 2:, -1]).all()
    out, state = kda.recurrence_prefill(x, i["la"], -math.inf, state_in=i["s0"])
    step = [kda.recurrence_step(x[:, t].contiguous(), i["la"][:, t].contiguous(), s, -math.inf)
            for s in [i["s0"].clone()] for t in range(min(T, 20))]
    torch.cuda.synchronize()
    same_where_not_finite(out, want["out"], "out")
    same_where_not_finite(state, want["state"], "state")
    same_where_not_finite(torch.stack(step, 1), want["out"][:, :20], "step")
    # the gradient runs the same recurrence in the other direction
    i["s0"][1] = 1.0
    want = run(i["x"], d)
    assert torch.isinf(want["dx"][:, :-2, :-1]).all()
    _, _, ws = kda.recurrence_prefill_for_backward(i["x"], i["la"], -math.inf, state_in=i["s0"])
    r = kda.recurrence_backward(i["x"], i["la"], -math.inf, ws, state_in=i["s0"], d_out=d, d_state=i["d_state"])
    torch.cuda.synchronize()
    for k in ("dx", "dlog_alpha", "dstate0"):
        same_where_not_finite(r[k], want[k], k)


@pytest.mark.parametrize("D", [3, 130])
@pytest.mark.parametrize("many", [1, 2, 1 << 19])
def test_any_number_of_empty_sequences(many, D):
    """Wherever they lie they pass their states through, and the others are what they are without them."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    ends, T = [0, 5, 130, 131, 500, 700], 700
    i = made(1, T, D, "f32", n=len(ends) - 1)
    full = []                                             # offsets with `many` empty ones in front of four of the sequences and behind the last
    for k, e in enumerate(ends):
        full += [e] * (1 + (many if k in (0, 1, 2, 4, 5) else 0))
    full = i32(full)
    held = (full.diff() > 0).nonzero()[:, 0]              # the sequences that have tokens
    assert len(held) == len(ends) - 1 and len(full) == len(ends) + 5 * many

    def go(cu, s0, ds):
        out, state, ws = kda.recurrence_prefill_for_backward(i["x"], i["la"], FLOOR, g=i["g"], state_in=s0, cu_seqlens=cu)
        r = kda.recurrence_backward(i["x"], i["la"], FLOOR, ws, g=i["g"], state_in=s0, cu_seqlens=cu, d_out=i["d_out"], d_state=ds)
        return [out, r["dx"], r["dlog_alpha"], r["dg"]], [state, r["dstate0"]]

    s0, ds = (torch.randn(len(full) - 1, D, device="cuda") for _ in range(2))
    s0[held], ds[held] = i["s0"], i["d_state"]
    rows, states = go(full, s0, ds)
    want_rows, want_states = go(i32(ends), i["s0"], i["d_state"])
    torch.cuda.synchronize()
    for a, b in zip(rows, want_rows):
        assert torch.equal(a, b)
    for got, want, before in zip(states, want_states, (s0, ds)):
        expected = before.clone()
        expected[held] = want
        assert torch.equal(got, expected)
