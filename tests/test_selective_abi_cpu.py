"""The short convolution and the selective scan through the C ABI, without a
GPU: the header, the exports and the binding agree, and bad arguments are
refused before anything touches a device."""
import ctypes
import os
import re

import pytest

import gated_delta_rule_91_amd as kda
from gated_delta_rule_91_amd import selective

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kda_selective.h")
FAKE = 0x10000            # aligned, never dereferenced: validation fails first
MISALIGNED = 0x10008
BAD, UNSUPPORTED, SMALL = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_91_amd import build
        build.build()
    return selective._slib()


def test_exports_every_declared_symbol(L):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(kda_[a-z0-9_]+)\s*\(", src)))
    assert sorted(kda.SELECTIVE_EXPORTS) == names
    for n in names:
        assert getattr(L, n).argtypes is not None, n
    assert not set(names) & (set(kda.EXPORTS) | set(kda.HYBRID_EXPORTS))
    for n in selective.__all__:
        assert getattr(kda, n) is getattr(selective, n)


def conv(**kw):
    base = dict(batch=2, seqlen=50, width=20, n_seq=-1, taps=4, silu=1, io_dtype=kda.KDA_BF16)
    base.update(kw)
    return selective.KdaShortConvProblem(*[base[n] for n, _ in selective.KdaShortConvProblem._fields_])


BAD_ROWS = [dict(batch=-1), dict(seqlen=-1), dict(width=0), dict(width=-4), dict(n_seq=-2), dict(n_seq=3), dict(io_dtype=2), dict(io_dtype=-1)]
LARGE_ROWS = [dict(seqlen=2 ** 30 + 1), dict(width=2 ** 30 + 1), dict(batch=2 ** 24 + 1), dict(batch=1, n_seq=2 ** 24 + 1),
              dict(batch=2 ** 20, seqlen=2 ** 20, width=2)]
BAD_CONV = BAD_ROWS + [dict(taps=0), dict(taps=-1), dict(silu=2), dict(silu=-1)]
LARGE_CONV = LARGE_ROWS + [dict(taps=1), dict(taps=5), dict(batch=1, seqlen=0, width=2 ** 30), dict(batch=1, n_seq=2 ** 24, seqlen=4, width=2 ** 20)]


def test_conv_refusals(L):
    names = ["p", "x", "weight", "bias", "state_in", "cu", "out", "state_out"]
    base = dict(p=conv(), x=FAKE, weight=FAKE, bias=FAKE, state_in=FAKE, cu=None, out=2 * FAKE, state_out=FAKE)
    call = lambda **kw: L.kda_short_conv_prefill(*[{**base, **kw}[n] for n in names], None)
    for kw in BAD_CONV:
        assert call(p=conv(**kw)) == BAD, kw
    for kw in LARGE_CONV:
        assert call(p=conv(**kw)) == UNSUPPORTED, kw
    for kw in (dict(p=None), dict(x=None), dict(weight=None), dict(out=None), dict(x=MISALIGNED), dict(weight=MISALIGNED), dict(bias=MISALIGNED),
               dict(state_in=MISALIGNED), dict(out=MISALIGNED), dict(state_out=MISALIGNED), dict(cu=FAKE), dict(out=FAKE)):
        assert call(**kw) == BAD, kw
    packed = conv(batch=1, n_seq=3)
    for kw in (dict(cu=None), dict(cu=0x10002)):
        assert call(p=packed, **kw) == BAD, kw
    assert call(p=conv(batch=1, n_seq=0), cu=FAKE) == 0
    assert call(p=conv(seqlen=0), state_out=None) == 0
    assert call(p=conv(batch=0)) == 0 or call(p=conv(batch=0), state_out=None) == 0


def test_conv_backward_refusals(L):
    names = ["p", "x", "weight", "bias", "state_in", "cu", "d_out", "d_state", "dx", "dweight", "dbias", "d_state_in", "ws", "bytes"]
    need = L.kda_short_conv_backward_workspace_size(conv())
    assert need >= 2 * 5 * 20 * 4
    base = dict(p=conv(), x=FAKE, weight=FAKE, bias=FAKE, state_in=FAKE, cu=None, d_out=FAKE, d_state=FAKE, dx=2 * FAKE, dweight=FAKE, dbias=FAKE,
                d_state_in=FAKE, ws=FAKE, bytes=need)
    call = lambda **kw: L.kda_short_conv_backward(*[{**base, **kw}[n] for n in names], None)
    for kw in BAD_CONV:
        assert call(p=conv(**kw)) == BAD, kw
        assert L.kda_short_conv_backward_workspace_size(conv(**kw)) == 0
    for kw in LARGE_CONV:
        assert call(p=conv(**kw)) == UNSUPPORTED, kw
        assert L.kda_short_conv_backward_workspace_size(conv(**kw)) == 0
    for kw in (dict(p=None), dict(x=None), dict(weight=None), dict(dx=None), dict(dweight=None), dict(dbias=None), dict(ws=None), dict(cu=FAKE),
               dict(x=MISALIGNED), dict(weight=MISALIGNED), dict(bias=MISALIGNED), dict(state_in=MISALIGNED), dict(d_out=MISALIGNED),
               dict(d_state=MISALIGNED), dict(dx=MISALIGNED), dict(dweight=MISALIGNED), dict(dbias=MISALIGNED), dict(d_state_in=MISALIGNED),
               dict(ws=MISALIGNED), dict(dx=FAKE), dict(x=4 * FAKE, dx=4 * FAKE)):
        assert call(**kw) == BAD, kw
    assert call(bytes=need - 1) == SMALL
    assert L.kda_short_conv_backward_workspace_size(None) == 0


def test_conv_step_refusals(L):
    names = ["N", "D", "taps", "silu", "io", "x", "weight", "bias", "state", "out"]
    base = dict(N=3, D=20, taps=4, silu=1, io=kda.KDA_F32, x=FAKE, weight=FAKE, bias=FAKE, state=FAKE, out=FAKE)
    call = lambda **kw: L.kda_short_conv_step(*[{**base, **kw}[n] for n in names], None)
    for kw in (dict(N=-1), dict(D=0), dict(taps=0), dict(silu=3), dict(io=2), dict(x=None), dict(weight=None), dict(state=None), dict(out=None),
               dict(x=MISALIGNED), dict(weight=MISALIGNED), dict(bias=MISALIGNED), dict(state=MISALIGNED), dict(out=MISALIGNED)):
        assert call(**kw) == BAD, kw
    for kw in (dict(taps=1), dict(taps=5), dict(N=2 ** 20, D=2 ** 12), dict(N=2 ** 62, D=2 ** 62)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(N=0, x=None, weight=None, state=None, out=None) == 0


def scan(**kw):
    base = dict(batch=2, seqlen=500, width=20, n_seq=-1, states=16, io_dtype=kda.KDA_BF16)
    base.update(kw)
    return selective.KdaSelectiveScanProblem(*[base[n] for n, _ in selective.KdaSelectiveScanProblem._fields_])


def inputs(**kw):
    base = dict(x=FAKE, dt=FAKE, A=FAKE, B=FAKE, C=FAKE, skip=FAKE, z=FAKE, dt_bias=FAKE, state_in=FAKE, cu_seqlens=None)
    base.update(kw)
    return selective.KdaSelectiveScanInputs(*[base[n] for n, _ in selective.KdaSelectiveScanInputs._fields_])


def gradients(**kw):
    base = {n: FAKE for n, _ in selective.KdaSelectiveScanGradients._fields_}
    base.update(kw)
    return selective.KdaSelectiveScanGradients(*base.values())


BAD_SCAN = BAD_ROWS + [dict(states=0), dict(states=-8)]
LARGE_SCAN = LARGE_ROWS + [dict(states=1), dict(states=12), dict(states=64), dict(batch=2 ** 24, seqlen=2 ** 14, width=1), dict(batch=1, n_seq=2 ** 24, seqlen=4, width=2 ** 20)]
BAD_INPUTS = [{n: None} for n in ("x", "dt", "A", "B", "C")] + [{n: MISALIGNED} for n in ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias", "state_in")] + [dict(cu_seqlens=FAKE)]


@pytest.mark.parametrize("back", [False, True])
def test_scan_refusals(L, back):
    f = L.kda_selective_scan_prefill_for_backward if back else L.kda_selective_scan_prefill
    size = L.kda_selective_scan_backward_workspace_size if back else L.kda_selective_scan_workspace_size
    need = size(scan())
    assert need > 0
    call = lambda p=scan(), i=inputs(), out=FAKE, state=FAKE, ws=FAKE, n=need: f(p, i, out, state, ws, n, None)
    for kw in BAD_SCAN:
        assert call(p=scan(**kw)) == BAD and size(scan(**kw)) == 0, kw
    for kw in LARGE_SCAN:
        assert call(p=scan(**kw)) == UNSUPPORTED and size(scan(**kw)) == 0, kw
    for kw in BAD_INPUTS:
        assert call(i=inputs(**kw)) == BAD, kw
    for kw in (dict(p=None), dict(i=None), dict(out=None), dict(out=MISALIGNED), dict(state=MISALIGNED), dict(ws=None), dict(ws=MISALIGNED)):
        assert call(**kw) == BAD, kw
    assert call(n=need - 1) == SMALL
    packed = scan(batch=1, n_seq=3)
    assert call(p=packed) == BAD and call(p=packed, i=inputs(cu_seqlens=0x10002)) == BAD
    assert size(packed) > 0 and call(p=packed, i=inputs(cu_seqlens=FAKE), n=size(packed) - 1) == SMALL
    assert call(p=scan(batch=1, n_seq=0), i=inputs(cu_seqlens=FAKE), n=1 << 40) == 0
    assert call(p=scan(seqlen=0), state=None) == 0


def test_scan_backward_refusals(L):
    need = L.kda_selective_scan_backward_workspace_size(scan())
    call = lambda p=scan(), i=inputs(), go=FAKE, gs=FAKE, to=gradients(), ws=FAKE, n=need: L.kda_selective_scan_backward(p, i, go, gs, to, ws, n, None)
    for kw in BAD_SCAN:
        assert call(p=scan(**kw)) == BAD, kw
    for kw in LARGE_SCAN:
        assert call(p=scan(**kw)) == UNSUPPORTED, kw
    for kw in BAD_INPUTS:
        assert call(i=inputs(**kw)) == BAD, kw
    for n, _ in selective.KdaSelectiveScanGradients._fields_:
        assert call(to=gradients(**{n: MISALIGNED})) == BAD, n
        if n != "d_state_in":
            assert call(to=gradients(**{n: None})) == BAD, n
    for kw in (dict(p=None), dict(i=None), dict(to=None), dict(go=MISALIGNED), dict(gs=MISALIGNED), dict(ws=None), dict(ws=MISALIGNED)):
        assert call(**kw) == BAD, kw
    assert call(n=need - 1) == SMALL


def test_scan_step_refusals(L):
    names = ["N", "D", "states", "io", "x", "dt", "A", "B", "C", "skip", "z", "bias", "state", "out"]
    base = dict(N=3, D=20, states=16, io=kda.KDA_F32, **{n: FAKE for n in names[4:]})
    call = lambda **kw: L.kda_selective_scan_step(*[{**base, **kw}[n] for n in names], None)
    for kw in [dict(N=-1), dict(D=0), dict(states=0), dict(io=2)] + [{n: None} for n in ("x", "dt", "A", "B", "C", "state", "out")] + [{n: MISALIGNED} for n in names[4:]]:
        assert call(**kw) == BAD, kw
    for kw in (dict(states=4), dict(states=24), dict(N=2 ** 20, D=2 ** 12), dict(N=2 ** 62, D=2 ** 62)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(N=0, **{n: None for n in names[4:]}) == 0


def test_binding_checks_tensors():
    torch = pytest.importorskip("torch")
    t = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)
    x, w = t(2, 5, 8), t(8, 4)
    with pytest.raises(ValueError, match="on the GPU"):
        kda.short_conv_prefill(x, w)
    for args, kw in (((t(5, 8), w), {}), ((x, t(8, 5)), {}), ((x, t(7, 4)), {}), ((x, w), dict(bias=t(7))), ((x, w), dict(state_in=t(2, 4, 8))),
                     ((x, w.double()), {}), ((x.double(), w), {}), ((x.transpose(0, 1), w), {}), ((x, w), dict(cu_seqlens=torch.tensor([0, 5], dtype=torch.int32))),
                     ((x, w), dict(bias=t(8, dtype=torch.bfloat16)))):
        with pytest.raises((ValueError, TypeError)):
            kda.short_conv_prefill(*args, **kw)
        with pytest.raises((ValueError, TypeError)):
            kda.short_conv_backward(*args, **kw)
    with pytest.raises((ValueError, TypeError)):
        kda.short_conv_step(t(2, 8), w, t(2, 4, 8))
    with pytest.raises((ValueError, TypeError)):
        kda.short_conv_step(x, w, t(2, 3, 8))
    A, B = t(8, 16), t(2, 5, 16)
    with pytest.raises(ValueError, match="on the GPU"):
        kda.selective_scan_prefill(x, x, A, B, B, workspace=t(4, dtype=torch.uint8))
    for args, kw in (((t(5, 8), x, A, B, B), {}), ((x, t(2, 5, 7), A, B, B), {}), ((x, x, t(8, 12), B, B), {}), ((x, x, t(7, 16), B, B), {}),
                     ((x, x, A, t(2, 5, 8), B), {}), ((x, x, A, B, B.bfloat16()), {}), ((x, x, A, B, B), dict(z=t(2, 5, 9))),
                     ((x, x, A, B, B), dict(skip=t(9))), ((x, x, A, B, B), dict(dt_bias=t(8, 1))), ((x, x, A, B, B), dict(state_in=t(2, 8, 8))),
                     ((x, x, A, B, B), dict(cu_seqlens=torch.tensor([0, 5], dtype=torch.int32)))):
        with pytest.raises((ValueError, TypeError)):
            kda.selective_scan_prefill(*args, **kw)
        with pytest.raises((ValueError, TypeError)):
            kda.selective_scan_backward(*args, t(4, dtype=torch.uint8), **kw)
    with pytest.raises((ValueError, TypeError)):
        kda.selective_scan_step(t(2, 8), t(2, 8), A, t(2, 16), t(2, 16), t(2, 8, 8))


def test_problem_constructors():
    torch = pytest.importorskip("torch")
    p = kda.short_conv_problem(1, 1000, 64, 4, torch.bfloat16, n_seq=3)
    assert (p.n_seq, p.silu, p.io_dtype) == (3, 1, kda.KDA_BF16) and kda.short_conv_backward_workspace_size(p) > 0
    q = kda.selective_scan_problem(1, 1000, 64, 16, torch.float32, n_seq=3)
    assert kda.selective_scan_backward_workspace_size(q) > kda.selective_scan_workspace_size(q) > 0
    assert kda.selective_scan_workspace_size(kda.selective_scan_problem(1, 16, 64, 16, torch.float32)) == 0
    assert ctypes.sizeof(selective.KdaShortConvProblem) == 48 and ctypes.sizeof(selective.KdaSelectiveScanProblem) == 40


def test_shared_attention_refusals(L):
    from gated_delta_rule_91_amd import hybrid
    H = hybrid._hlib()
    cache = hybrid.KdaCache4(9, 64, 2, 128, FAKE, FAKE, FAKE, FAKE)
    problem = lambda **kw: hybrid.KdaCache4AttentionProblem(*{**dict(n_seq=3, tokens=3, heads=8, max_pages=6, max_q=1, max_len=384, io_dtype=kda.KDA_BF16, scale=0.1), **kw}.values())
    size = lambda p=None, n=2, most=100: H.kda_cache4_shared_attention_workspace_size(cache, p or problem(), n, most)
    names = ["q", "table", "total", "n", "prefix", "offsets", "most", "cu", "g", "out", "ws"]
    base = dict(q=FAKE, table=FAKE, total=FAKE, n=2, prefix=FAKE, offsets=FAKE, most=100, cu=None, g=None, out=2 * FAKE, ws=FAKE)
    call = lambda p=None, nbytes=1 << 40, **kw: H.kda_cache4_shared_attention(cache, p or problem(), *[{**base, **kw}[k] for k in names], nbytes, None)
    for kw in (dict(n_seq=-1), dict(heads=7), dict(max_q=0), dict(max_len=-1), dict(io_dtype=5), dict(scale=float("nan")), dict(tokens=4)):
        assert call(p=problem(**kw)) == BAD, kw
    for kw in (dict(n=-1), dict(most=-1), dict(q=None), dict(q=MISALIGNED), dict(table=None), dict(total=None), dict(prefix=None), dict(offsets=None),
               dict(prefix=0x10002), dict(offsets=0x10001), dict(cu=0x10002), dict(g=MISALIGNED), dict(out=None), dict(ws=None), dict(ws=MISALIGNED), dict(out=FAKE)):
        assert call(**kw) == BAD, kw
    for kw in (dict(n=2 ** 23 + 1), dict(n=2 ** 40)):
        assert call(**kw) == UNSUPPORTED and size(n=kw["n"]) == 0, kw
    for kw in (dict(n_seq=2 ** 25, tokens=2 ** 25), dict(max_pages=2 ** 26)):
        assert call(p=problem(**kw)) == UNSUPPORTED and size(problem(**kw)) == 0, kw
    assert size() > 0 and call(nbytes=size() - 1) == SMALL and size(n=-1) == 0 and size(most=-1) == 0
    assert size(n=0) == H.kda_cache4_attention_workspace_size(cache, problem())
    assert call(p=problem(n_seq=0, tokens=0), q=None, table=None, total=None, out=None, ws=None, nbytes=0) == 0


def test_shared_attention_binding_checks_tensors():
    torch = pytest.importorskip("torch")
    i32 = torch.int32
    t = lambda *s, dtype=i32: torch.zeros(*s, dtype=dtype)
    cache = kda.Cache4.empty(4, 16, 2, 64, device="cpu")
    q = t(3, 4, 64, dtype=torch.float32)
    for args in ((t(3, 2), t(3), t(2, 1), t(3)), (t(3, 2), t(3), t(2), t(2)), (t(3, 2), t(3), t(2), t(3, dtype=torch.int64)), (t(3, 2), t(2), t(2), t(3)),
                 (t(3, 2), t(3), t(2, dtype=torch.float32), t(3)), (t(3, 2), t(3), t(2), t(3))):       # the last: not on a GPU
        with pytest.raises((ValueError, TypeError)):
            kda.cache4_shared_attention(q, cache, *args)
