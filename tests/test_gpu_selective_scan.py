"""The selective scan on an MI355X against a plain 64-bit form, whose bounds
(tests/_selective_ref.py) are what its roundings in 32 bits can add up to; a
stored result is off by half a step of its type more."""
import math

import pytest

import _selective_ref as ref

torch = pytest.importorskip("torch")
import gated_delta_rule_91_amd as kda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
UO = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
MARK = 55.0
INPUTS = ("x", "dt", "A", "B", "C")
GIVEN = ("skip", "z", "dt_bias")


def made(R, T, D, N, io, n=None, skip=True, z=True, bias=True, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + R * 7 + T * 3 + D + N)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    n = R if n is None else n
    step = torch.exp(torch.rand(D, generator=gen, device="cuda") * math.log(300) + math.log(0.001))
    return dict(x=r(R, T, D).to(DT[io]), dt=r(R, T, D).to(DT[io]), A=-torch.arange(1, N + 1, device="cuda") * torch.exp(0.3 * r(D, N)),
                B=r(R, T, N).to(DT[io]), C=r(R, T, N).to(DT[io]), skip=r(D) if skip else None, z=r(R, T, D).to(DT[io]) if z else None,
                dt_bias=step + torch.log(-torch.expm1(-step)) if bias else None, state=r(n, D, N), d_out=r(R, T, D).to(DT[io]), d_state=r(n, D, N))


def within(got, want, label):
    value, bound = want
    keep = ~torch.isnan(value)
    tol = bound + UO[got.dtype] * value.abs() + 1e-37
    worst = ((got.cpu().double() - value).abs() / tol)[keep]
    assert got.shape == value.shape
    assert worst.numel() == 0 or float(worst.max()) <= 1, (label, float(worst.max()))


def call(i, cut, **kw):
    return [i[k] for k in INPUTS], dict({k: i[k] for k in GIVEN}, state_in=i["state"], cu_seqlens=cut, **kw)


def check(i, cu=None, backward=True):
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    cpu = {k: None if v is None else v.cpu() for k, v in i.items()}
    want = ref.scan(*(cpu[k] for k in INPUTS), *(cpu[k] for k in GIVEN), cpu["state"], cu, *((cpu["d_out"], cpu["d_state"]) if backward else ()))
    room = torch.full((i["x"].numel() + 64,), MARK, dtype=i["x"].dtype, device="cuda")
    out = room[:i["x"].numel()].view(i["x"].shape)
    args, kw = call(i, cut)
    _, state = kda.selective_scan_prefill(*args, **kw, out=out)
    torch.cuda.synchronize()
    assert (room[i["x"].numel():] == MARK).all()
    left = torch.isnan(want["out"][0])
    assert (out.cpu()[left] == MARK).all()                # tokens of no sequence
    within(out, want["out"], "out")
    within(state, want["state"], "state")
    # the state in place
    kept = i["state"].clone()
    out1, _ = kda.selective_scan_prefill(*args, **dict(kw, state_in=kept), state_out=kept)
    torch.cuda.synchronize()
    assert torch.equal(out1.cpu()[~left], out.cpu()[~left]) and torch.equal(kept, state)
    if not backward:
        return
    out2, state2, ws = kda.selective_scan_prefill_for_backward(*args, **kw)
    torch.cuda.synchronize()
    assert torch.equal(out2.cpu()[~left], out.cpu()[~left]) and torch.equal(state2, state)
    first = None
    for _ in range(2):                                    # the workspace serves a second call
        r = kda.selective_scan_backward(*args, ws, **kw, d_out=i["d_out"], d_state=i["d_state"])
        torch.cuda.synchronize()
        for name in ("dx", "ddt", "dA", "dB", "dC", "dstate0") + tuple(g for g, k in (("dskip", "skip"), ("dz", "z"), ("ddt_bias", "dt_bias")) if i[k] is not None):
            within(r[name], want[name], name)
        for g, k in (("dskip", "skip"), ("dz", "z"), ("ddt_bias", "dt_bias")):
            assert (r[g] is None) == (i[k] is None)
        if first is not None:
            assert all(v is None or torch.equal(torch.nan_to_num(v[..., :0].float() if cu else v.float()), torch.nan_to_num(first[k][..., :0].float() if cu else first[k].float()))
                       for k, v in r.items())
        first = r


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("R,T,D", [(1, 1, 1), (2, 3, 5), (1, 16, 64), (1, 33, 65), (3, 64, 7), (2, 100, 130), (1, 257, 20)])
def test_uniform(R, T, D, N, io):
    check(made(R, T, D, N, io))


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_uniform_long(io):
    check(made(1, 1500, 66, 16, io))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("skip,z,bias", [(False, False, False), (True, False, False), (False, True, False), (False, False, True)])
def test_what_may_be_left_out(skip, z, bias, io):
    check(made(2, 70, 66, 16, io, skip=skip, z=z, bias=bias))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("cu,T,D", [([0, 5], 5, 3), ([0, 1, 2, 3], 3, 64), ([0, 32, 64], 64, 66), ([0, 0, 40, 40, 40, 170, 170], 170, 33),
                                    ([0, 31, 32, 33, 65, 200], 200, 20), ([3, 10, 80], 120, 64), ([0, 0], 40, 8), ([40, 40], 40, 8), ([50, 60], 60, 5),
                                    ([2, 100, 100, 125], 130, 65)])
def test_packed(cu, T, D, N, io):
    check(made(1, T, D, N, io, n=len(cu) - 1), cu=cu)


def test_packed_many_short_sequences():
    gen = torch.Generator().manual_seed(5)
    cu = [0]
    for m in torch.randint(0, 9, (200,), generator=gen).tolist():
        cu.append(cu[-1] + m)
    check(made(1, cu[-1], 70, 16, "f32", n=200), cu=cu)


def test_many_rows_and_one_tile():
    """Enough rows that time is not split."""
    check(made(1100, 20, 130, 8, "bf16"), backward=False)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_nothing_given(io):
    i = made(2, 50, 20, 8, io, skip=False, z=False, bias=False)
    args = [i[k] for k in INPUTS]
    want = ref.scan(*(i[k].cpu() for k in INPUTS), d_out=i["d_out"].cpu())
    out, state = kda.selective_scan_prefill(*args, want_state=False)
    _, _, ws = kda.selective_scan_prefill_for_backward(*args)
    r = kda.selective_scan_backward(*args, ws, d_out=i["d_out"], want_dstate=False)
    none = kda.selective_scan_backward(*args, ws)
    torch.cuda.synchronize()
    within(out, want["out"], "out")
    for k in ("dx", "ddt", "dA", "dB", "dC"):
        within(r[k], want[k], k)
    assert state is None and r["dstate0"] is None
    assert all(v is None or not v.any() for v in none.values())


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("n,D", [(1, 1), (3, 7), (5, 64), (2, 515), (257, 20)])
def test_step(n, D, N, io):
    i = made(n, 1, D, N, io, seed=3)
    want = ref.scan(*(i[k].cpu() for k in INPUTS + GIVEN), i["state"].cpu())
    state = i["state"].clone()
    one = {k: i[k][:, 0].contiguous() for k in ("x", "dt", "B", "C", "z")}
    out = kda.selective_scan_step(one["x"], one["dt"], i["A"], one["B"], one["C"], state, skip=i["skip"], z=one["z"], dt_bias=i["dt_bias"])
    torch.cuda.synchronize()
    within(out[:, None], want["out"], "out")
    within(state, want["state"], "state")


def test_steps_go_on_from_a_prompt():
    i = made(2, 60, 40, 16, "f32", seed=9)
    want = ref.scan(*(i[k].cpu() for k in INPUTS + GIVEN), i["state"].cpu())
    cut = lambda k, b, e: i[k][:, b:e].contiguous()
    head = {k: cut(k, 0, 50) for k in ("x", "dt", "B", "C", "z")}
    out, s = kda.selective_scan_prefill(head["x"], head["dt"], i["A"], head["B"], head["C"], skip=i["skip"], z=head["z"], dt_bias=i["dt_bias"], state_in=i["state"])
    outs = [out]
    for t in range(50, 60):
        one = {k: cut(k, t, t + 1)[:, 0].contiguous() for k in ("x", "dt", "B", "C", "z")}
        outs.append(kda.selective_scan_step(one["x"], one["dt"], i["A"], one["B"], one["C"], s, skip=i["skip"], z=one["z"], dt_bias=i["dt_bias"])[:, None])
    torch.cuda.synchronize()
    within(torch.cat(outs, 1), want["out"], "out")
    within(s, want["state"], "state")


def test_extremes_of_the_step_size():
    """delta from far below 2^-24 to beyond what exp(-delta) leaves, and A = 0: a state that does not fade."""
    i = made(1, 90, 64, 8, "f32", bias=False, seed=2)
    i["dt"][0, :, 0::4] = -30.0        # delta = 9e-14
    i["dt"][0, :, 1::4] = 80.0         # exp(-80) and less: nothing is left of the state before
    i["dt"][0, 40, 2::4] = -200.0      # delta = 0 in 32 bits: the token leaves the state as it is
    i["A"][3::4] = 0.0
    check(i)
    i["dt"][0, :, 0::4] = -float("inf")
    args, kw = call(i, None)
    out, state = kda.selective_scan_prefill(*args, **kw)
    torch.cuda.synchronize()
    assert torch.equal(state[:, 0::4], i["state"][:, 0::4]) and torch.isfinite(out).all()


def test_autograd():
    gen = torch.Generator(device="cuda").manual_seed(4)
    i = made(1, 60, 12, 8, "f32", n=3, seed=6)
    cu = [2, 9, 9, 51]
    leaves = {k: i[k].clone().requires_grad_() for k in INPUTS + GIVEN + ("state",)}
    out, state = kda.selective_scan_autograd(*(leaves[k] for k in INPUTS + GIVEN + ("state",)), torch.tensor(cu, dtype=torch.int32, device="cuda"))
    ((out * i["d_out"]).sum() + (state * i["d_state"]).sum()).backward()
    want = ref.scan(*(i[k].cpu() for k in INPUTS + GIVEN + ("state",)), cu, i["d_out"].cpu(), i["d_state"].cpu())
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", skip="dskip", z="dz", dt_bias="ddt_bias", state="dstate0")
    for k, t in leaves.items():
        within(t.grad, want[names[k]], names[k])
    for k in ("x", "dt", "B", "C", "z"):
        assert not leaves[k].grad[0, :2].any() and not leaves[k].grad[0, 51:].any()
    assert not out[0, :2].any() and not out[0, 51:].any()
    del gen


def test_differences():
    """The gradient of a scalar loss against central differences of the 64-bit form."""
    i = made(1, 14, 3, 8, "f32", seed=8)
    names = INPUTS + GIVEN + ("state",)
    cpu = {k: v.cpu().double() for k, v in i.items()}
    args, kw = call(i, None)
    _, _, ws = kda.selective_scan_prefill_for_backward(*args, **kw)
    r = kda.selective_scan_backward(*args, ws, **kw, d_out=i["d_out"], d_state=i["d_state"])
    torch.cuda.synchronize()

    def loss(**change):
        v = {**cpu, **change}
        f = ref.scan(*(v[k] for k in names))
        return float((f["out"][0] * cpu["d_out"]).sum() + (f["state"][0] * cpu["d_state"]).sum())

    h = 1e-5        # central differences are off by h^2 / 6 of a third derivative, some 1e-9 here, and 1e-16 / h of the loss
    grads = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", skip="dskip", z="dz", dt_bias="ddt_bias", state="dstate0")
    for name in names:
        flat = cpu[name].flatten()
        for k in range(0, flat.numel(), max(1, flat.numel() // 5)):
            e = torch.zeros_like(flat)
            e[k] = h
            e = e.view(cpu[name].shape)
            d = (loss(**{name: cpu[name] + e}) - loss(**{name: cpu[name] - e})) / (2 * h)
            g = float(r[grads[name]].flatten()[k])
            assert abs(d - g) <= 1e-5 * (1 + abs(d)), (name, k, d, g)
