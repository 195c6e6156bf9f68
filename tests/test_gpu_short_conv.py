"""The short causal convolution on an MI355X against a plain 64-bit form, whose
bounds (tests/_selective_ref.py) are what its roundings in 32 bits can add up to;
a stored result is off by half a step of its type more."""
import pytest

import _selective_ref as ref

torch = pytest.importorskip("torch")
import gated_delta_rule_91_amd as kda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
UO = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
MARK = 55.0


def made(B, T, D, W, io, n=None, bias=True, seed=0, d_state=True):
    gen = torch.Generator(device="cuda").manual_seed(seed + B * 7 + T * 3 + D + W)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    n = B if n is None else n
    return dict(x=r(B, T, D).to(DT[io]), weight=r(D, W), bias=r(D) if bias else None, state=r(n, W - 1, D).to(DT[io]),
                d_out=r(B, T, D).to(DT[io]), d_state=r(n, W - 1, D).to(DT[io]) if d_state else None)


def within(got, want, label):
    value, bound = want
    keep = ~torch.isnan(value)
    tol = bound + UO[got.dtype] * value.abs() + 1e-37
    worst = ((got.cpu().double() - value).abs() / tol)[keep]
    assert got.shape == value.shape
    assert worst.numel() == 0 or float(worst.max()) <= 1, (label, float(worst.max()))


def marked(like):
    """Room for a result with a margin behind it, all of it marked."""
    room = torch.full((like.numel() + 64,), MARK, dtype=like.dtype, device="cuda")
    return room, room[:like.numel()].view(like.shape)


def check(i, silu, cu=None):
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    cpu = {k: None if v is None else v.cpu() for k, v in i.items()}
    want = ref.conv(cpu["x"], cpu["weight"], cpu["bias"], silu, cpu["state"], cu, cpu["d_out"], cpu["d_state"])
    room, out = marked(i["x"])
    got, state = kda.short_conv_prefill(i["x"], i["weight"], i["bias"], silu=silu, state_in=i["state"], cu_seqlens=cut, out=out)
    torch.cuda.synchronize()
    assert (room[i["x"].numel():] == MARK).all()
    left = torch.isnan(want["out"][0])
    assert (out.cpu()[left] == MARK).all()                # tokens of no sequence
    within(out, want["out"], "out")
    assert torch.equal(state.cpu().double(), want["state"][0])
    r = kda.short_conv_backward(i["x"], i["weight"], i["d_out"], bias=i["bias"], silu=silu, state_in=i["state"], cu_seqlens=cut, d_state=i["d_state"])
    torch.cuda.synchronize()
    for name in ("dx", "dweight", "dstate0"):
        within(r[name], want[name], name)
    if i["bias"] is None:
        assert r["dbias"] is None
    else:
        within(r["dbias"], want["dbias"], "dbias")
    # the state in place
    kept = i["state"].clone()
    out2, state2 = kda.short_conv_prefill(i["x"], i["weight"], i["bias"], silu=silu, state_in=kept, state_out=kept, cu_seqlens=cut)
    torch.cuda.synchronize()
    assert torch.equal(out2.cpu()[~left], out.cpu()[~left]) and torch.equal(kept, state)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("W,silu,bias", [(2, True, False), (3, False, True), (4, True, True)])
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (2, 2, 3), (3, 5, 4), (2, 17, 7), (1, 64, 8), (1, 65, 9), (2, 130, 64), (1, 67, 515), (3, 33, 1030)])
def test_uniform(B, T, D, W, silu, bias, io):
    check(made(B, T, D, W, io, bias=bias), silu)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("cu,T,D", [([0, 5], 5, 3), ([0, 1, 2, 3], 3, 16), ([0, 16, 32], 32, 24), ([0, 0, 20, 20, 20, 90, 90], 90, 13),
                                    ([3, 10, 50], 60, 32), ([0, 0], 40, 8), ([40, 40], 40, 8), ([2, 30, 30, 31, 33, 64, 65], 70, 65)])
def test_packed(cu, T, D, W, io):
    check(made(1, T, D, W, io, n=len(cu) - 1), True, cu=cu)


def test_packed_many_short_sequences():
    gen = torch.Generator().manual_seed(5)
    cu = [0]
    for m in torch.randint(0, 6, (300,), generator=gen).tolist():
        cu.append(cu[-1] + m)
    check(made(1, cu[-1], 70, 4, "bf16", n=300), True, cu=cu)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_nothing_given(io):
    """No bias, no state, no gradient of the state, and none of the output."""
    i = made(2, 40, 20, 4, io, bias=False, d_state=False)
    i["state"] = None
    check_ = dict(i, state=None)
    want = ref.conv(i["x"].cpu(), i["weight"].cpu(), None, True, None, None, i["d_out"].cpu(), None)
    out, state = kda.short_conv_prefill(i["x"], i["weight"], want_state=False)
    r = kda.short_conv_backward(i["x"], i["weight"], i["d_out"], want_dstate=False)
    none = kda.short_conv_backward(i["x"], i["weight"])
    torch.cuda.synchronize()
    within(out, want["out"], "out")
    within(r["dx"], want["dx"], "dx")
    within(r["dweight"], want["dweight"], "dweight")
    assert state is None and r["dstate0"] is None and check_["bias"] is None
    assert not none["dx"].any() and not none["dweight"].any() and not none["dstate0"].any()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("N,D", [(1, 1), (3, 7), (5, 8), (2, 515), (257, 64)])
def test_step(N, D, W, io):
    i = made(N, 1, D, W, io, seed=3)
    want = ref.conv(i["x"].cpu(), i["weight"].cpu(), i["bias"].cpu(), True, i["state"].cpu())
    state = i["state"].clone()
    out = kda.short_conv_step(i["x"][:, 0].contiguous(), i["weight"], state, bias=i["bias"])
    torch.cuda.synchronize()
    within(out[:, None], want["out"], "out")
    assert torch.equal(state.cpu().double(), want["state"][0])


@pytest.mark.parametrize("silu", [True, False])
def test_steps_go_on_from_a_prompt(silu):
    """A prompt, then token by token: the same bits as the whole at once (the sums are taken in the same order)."""
    i = made(3, 50, 40, 4, "f32", seed=9)
    whole, state = kda.short_conv_prefill(i["x"], i["weight"], i["bias"], silu=silu, state_in=i["state"])
    head, s = kda.short_conv_prefill(i["x"][:, :41].contiguous(), i["weight"], i["bias"], silu=silu, state_in=i["state"])
    outs = [kda.short_conv_step(i["x"][:, t].contiguous(), i["weight"], s, bias=i["bias"], silu=silu) for t in range(41, 50)]
    torch.cuda.synchronize()
    assert torch.equal(torch.cat([head, torch.stack(outs, 1)], 1), whole) and torch.equal(s, state)


def test_infinite_and_nan_inputs_stay_where_they_are():
    """An input that is no number reaches the taps behind it, of its own channel and sequence, and nothing else."""
    i = made(1, 40, 16, 4, "f32", n=2)
    i["x"][0, 9, 3], i["x"][0, 19, 5] = float("nan"), float("inf")
    out, _ = kda.short_conv_prefill(i["x"], i["weight"], silu=False, cu_seqlens=torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    odd = ~torch.isfinite(out[0].cpu())
    want = torch.zeros(40, 16, dtype=torch.bool)
    want[9:13, 3] = True
    want[19, 5] = True
    assert torch.equal(odd, want)


def test_autograd():
    gen = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    cu = torch.tensor([2, 9, 9, 31], dtype=torch.int32, device="cuda")
    x, w, b, s = (t.requires_grad_() for t in (r(1, 40, 12), r(12, 4), r(12), r(3, 3, 12)))
    out, state = kda.short_conv_autograd(x, w, b, True, s, cu)
    go, gs = r(1, 40, 12), r(3, 3, 12)
    (out * go).sum().backward(retain_graph=True)
    (state * gs).sum().backward()
    want = ref.conv(*(t.detach().cpu() for t in (x, w, b)), True, s.detach().cpu(), cu.tolist(), go.cpu(), gs.cpu())
    assert not out[0, :2].any() and not out[0, 31:].any() and not x.grad[0, :2].any() and not x.grad[0, 31:].any()
    for t, n in ((x, "dx"), (w, "dweight"), (b, "dbias"), (s, "dstate0")):
        value, bound = want[n]
        keep = ~torch.isnan(value)
        # two passes, whose gradients are added
        assert ((t.grad.cpu().double() - value).abs() <= 2 * bound + 4 * 2.0 ** -24 * value.abs() + 1e-6 * (1 + value.abs()))[keep].all(), n


def test_differences():
    """The gradient of a scalar loss against central differences of the 64-bit form."""
    i = made(1, 12, 3, 4, "f32", seed=8)
    cpu = {k: v.cpu().double() for k, v in i.items()}
    r = kda.short_conv_backward(i["x"], i["weight"], i["d_out"], bias=i["bias"], state_in=i["state"], d_state=i["d_state"])
    torch.cuda.synchronize()

    def loss(**kw):
        v = {**cpu, **kw}
        f = ref.conv(v["x"], v["weight"], v["bias"], True, v["state"])
        return float((f["out"][0] * cpu["d_out"]).sum() + (f["state"][0] * cpu["d_state"]).sum())

    h = 1e-5        # central differences are off by h^2 / 6 of a third derivative, some 1e-9 here, and 1e-16 / h of the loss
    for name, grad in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias"), ("state", "dstate0")):
        flat = cpu[name].flatten()
        for k in range(0, flat.numel(), max(1, flat.numel() // 7)):
            e = torch.zeros_like(flat)
            e[k] = h
            e = e.view(cpu[name].shape)
            d = (loss(**{name: cpu[name] + e}) - loss(**{name: cpu[name] - e})) / (2 * h)
            g = float(r[grad].flatten()[k])
            assert abs(d - g) <= 1e-5 * (1 + abs(d)), (name, k, d, g)
