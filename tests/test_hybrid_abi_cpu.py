"""The operators beside KDA through the C ABI, without a GPU: the header, the
exports and the binding agree, and bad arguments are refused before anything
touches a device."""
import ctypes
import os
import re

import pytest

import gated_delta_rule_91_amd as kda
from gated_delta_rule_91_amd import hybrid

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kda_hybrid.h")
FAKE = 0x10000            # aligned, never dereferenced: validation fails first
MISALIGNED = 0x10008
BAD, UNSUPPORTED, SMALL = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_91_amd import build
        build.build()
    return hybrid._hlib()


def test_exports_every_declared_symbol(L):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(kda_[a-z0-9_]+)\s*\(", src)))
    assert sorted(kda.HYBRID_EXPORTS) == names
    for n in names:
        assert hasattr(L, n), n
    assert not set(names) & set(kda.EXPORTS)


def test_plan_refusals(L):
    names = ["n", "tokens", "page", "width", "past", "new", "table", "n_free", "free", "cu", "total", "slots", "taken"]
    base = dict(n=3, tokens=10, page=64, width=4, past=FAKE, new=FAKE, table=FAKE, n_free=5, free=FAKE, cu=FAKE,
                total=FAKE, slots=FAKE, taken=FAKE)
    call = lambda **kw: L.kda_plan_requests(*[{**base, **kw}[n] for n in names], None)
    for kw in (dict(n=-1), dict(tokens=-1), dict(width=-1), dict(n_free=-1), dict(page=0), dict(page=8),
               dict(page=48), dict(page=512), dict(past=None), dict(new=None), dict(table=None), dict(free=None),
               dict(cu=None), dict(total=None), dict(slots=None), dict(taken=None), dict(slots=0x10004),
               dict(past=0x10002)):
        assert call(**kw) == BAD, kw
    for kw in (dict(n=8193), dict(tokens=2 ** 31), dict(n_free=2 ** 31), dict(n=8192, width=2 ** 18)):
        assert call(**kw) == UNSUPPORTED, kw


def cache(**kw):
    base = dict(pages=9, page_size=64, heads=2, d=128, k=FAKE, k_scale=FAKE, v=FAKE, v_scale=FAKE)
    base.update(kw)
    return hybrid.KdaCache4(*[base[n] for n, _ in hybrid.KdaCache4._fields_])


BAD_CACHES = [dict(pages=-1), dict(page_size=8), dict(page_size=0), dict(page_size=96), dict(heads=0), dict(d=0),
              dict(k=None), dict(k_scale=None), dict(v=MISALIGNED), dict(v_scale=0x10001)]


@pytest.mark.parametrize("name", ["kda_cache4_append", "kda_cache4_read"])
def test_cache_rows_refusals(L, name):
    f = getattr(L, name)
    call = lambda c=None, tokens=5, io=kda.KDA_BF16, k=FAKE, v=FAKE, s=FAKE: f(c or cache(), tokens, io, k, v, s, None)
    for kw in BAD_CACHES:
        assert call(c=cache(**kw)) == BAD, kw
    assert f(None, 5, kda.KDA_BF16, FAKE, FAKE, FAKE, None) == BAD
    assert call(c=cache(d=96)) == UNSUPPORTED
    assert call(c=cache(pages=2 ** 50)) == UNSUPPORTED
    assert call(tokens=2 ** 45) == UNSUPPORTED
    for kw in (dict(tokens=-1), dict(io=2), dict(k=None), dict(v=MISALIGNED), dict(s=None), dict(s=0x10004)):
        assert call(**kw) == BAD, kw
    assert call(tokens=0, k=None, v=None, s=None) == 0


def problem(**kw):
    base = dict(n_seq=3, tokens=3, heads=8, max_pages=6, max_q=1, max_len=384, io_dtype=kda.KDA_BF16, scale=0.1)
    base.update(kw)
    return hybrid.KdaCache4AttentionProblem(*[base[n] for n, _ in hybrid.KdaCache4AttentionProblem._fields_])


def test_attention_refusals(L):
    names = ["q", "table", "total", "cu", "g", "out", "ws"]
    base = dict(q=FAKE, table=FAKE, total=FAKE, cu=None, g=None, out=FAKE, ws=FAKE)

    def call(p=None, c=None, nbytes=1 << 40, **kw):
        return L.kda_cache4_attention(c or cache(), p or problem(), *[{**base, **kw}[n] for n in names], nbytes, None)

    for kw in BAD_CACHES:
        assert call(c=cache(**kw)) == BAD, kw
        assert L.kda_cache4_attention_workspace_size(cache(**kw), problem()) == 0
    for kw in (dict(n_seq=-1), dict(tokens=-1), dict(heads=0), dict(heads=7), dict(max_pages=-1), dict(max_q=0),
               dict(max_len=-1), dict(io_dtype=5), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert call(p=problem(**kw)) == BAD, kw
        assert L.kda_cache4_attention_workspace_size(cache(), problem(**kw)) == 0
    for kw in (dict(n_seq=2 ** 25, tokens=2 ** 25), dict(tokens=2 ** 29), dict(max_pages=2 ** 26)):
        assert call(p=problem(**kw)) == UNSUPPORTED, kw
    assert call(p=problem(tokens=4)) == BAD            # one row a sequence without offsets
    for kw in (dict(q=None), dict(q=MISALIGNED), dict(table=None), dict(total=None), dict(cu=0x10002),
               dict(g=MISALIGNED), dict(out=None)):
        assert call(**kw) == BAD, kw
    assert call(p=problem(n_seq=0, tokens=0), q=None, table=None, total=None, out=None, ws=None, nbytes=0) == 0
    # a long sequence is split: the partial results need a workspace
    p = problem(n_seq=1, tokens=1, max_pages=2048, max_len=131072)
    need = L.kda_cache4_attention_workspace_size(cache(), p)
    if need:
        assert call(p=p, nbytes=need - 1) == SMALL
        assert call(p=p, ws=None) == BAD


def rec(**kw):
    base = dict(batch=2, seqlen=300, width=130, n_seq=-1, io_dtype=kda.KDA_BF16, log_alpha_min=-0.5)
    base.update(kw)
    return hybrid.KdaRecurrenceProblem(*[base[n] for n, _ in hybrid.KdaRecurrenceProblem._fields_])


BAD_RECURRENCES = [dict(batch=-1), dict(seqlen=-1), dict(width=0), dict(n_seq=-2), dict(io_dtype=9),
                   dict(log_alpha_min=0.0), dict(log_alpha_min=float("nan")), dict(n_seq=3)]
LARGE_RECURRENCES = [dict(seqlen=2 ** 31), dict(width=2 ** 31), dict(batch=2 ** 25), dict(batch=1, n_seq=2 ** 25),
                     dict(batch=1, seqlen=2 ** 30, width=2 ** 20)]


@pytest.mark.parametrize("name", ["kda_recurrence_prefill", "kda_recurrence_prefill_for_backward"])
def test_recurrence_refusals(L, name):
    f = getattr(L, name)
    names = ["x", "la", "g", "s0", "cu", "out", "s1", "ws"]
    base = dict(x=FAKE, la=FAKE, g=None, s0=None, cu=None, out=FAKE, s1=FAKE, ws=FAKE)
    call = lambda p=None, nbytes=1 << 50, **kw: f(p or rec(), *[{**base, **kw}[n] for n in names], nbytes, None)
    assert f(None, *[base[n] for n in names], 1 << 50, None) == BAD
    for kw in BAD_RECURRENCES:
        assert call(p=rec(**kw), cu=FAKE if "n_seq" in kw else None) == BAD, kw
        assert L.kda_recurrence_workspace_size(rec(**kw)) == 0
        assert L.kda_recurrence_backward_workspace_size(rec(**kw)) == 0
    for kw in LARGE_RECURRENCES:
        assert call(p=rec(**kw), cu=FAKE if "n_seq" in kw else None) == UNSUPPORTED, kw
    for kw in (dict(x=None), dict(la=MISALIGNED), dict(g=MISALIGNED), dict(s0=MISALIGNED), dict(out=None),
               dict(s1=MISALIGNED), dict(cu=FAKE)):
        assert call(**kw) == BAD, kw
    assert call(p=rec(batch=1, n_seq=2), cu=None) == BAD
    assert call(p=rec(batch=1, n_seq=2), cu=0x10002) == BAD
    size = L.kda_recurrence_workspace_size if name == "kda_recurrence_prefill" else L.kda_recurrence_backward_workspace_size
    need = size(rec(seqlen=70000))
    if need:
        assert call(p=rec(seqlen=70000), nbytes=need - 1) == SMALL
        assert call(p=rec(seqlen=70000), ws=None) == BAD
    assert call(p=rec(batch=0), x=None, la=None, out=None, s1=None, ws=None, nbytes=0) == 0
    assert call(p=rec(seqlen=0), x=None, la=None, out=None, s1=None, ws=None, nbytes=0) == 0


def test_recurrence_backward_and_step_refusals(L):
    names = ["x", "la", "g", "s0", "cu", "do", "ds", "dx", "dla", "dg", "ds0", "ws"]
    base = {n: FAKE for n in names}
    base["cu"] = None
    call = lambda p=None, nbytes=1 << 50, **kw: L.kda_recurrence_backward(
        p or rec(), *[{**base, **kw}[n] for n in names], nbytes, None)
    for kw in BAD_RECURRENCES:
        assert call(p=rec(**kw), cu=FAKE if "n_seq" in kw else None) == BAD, kw
    for kw in LARGE_RECURRENCES:
        assert call(p=rec(**kw), cu=FAKE if "n_seq" in kw else None) == UNSUPPORTED, kw
    for kw in (dict(x=None), dict(la=None), dict(do=MISALIGNED), dict(ds=MISALIGNED), dict(dx=None), dict(dla=None),
               dict(dg=None), dict(ds0=MISALIGNED), dict(ws=None), dict(cu=FAKE)):
        assert call(**kw) == BAD, kw
    need = L.kda_recurrence_backward_workspace_size(rec())
    assert need > 0 and call(nbytes=need - 1) == SMALL
    step = lambda N=4, D=33, io=kda.KDA_F32, fl=-0.5, x=FAKE, la=FAKE, g=None, s=FAKE, o=FAKE: L.kda_recurrence_step(
        N, D, io, fl, x, la, g, s, o, None)
    for kw in (dict(N=-1), dict(D=0), dict(io=3), dict(fl=0.0), dict(x=None), dict(la=MISALIGNED), dict(g=MISALIGNED),
               dict(s=None), dict(o=None)):
        assert step(**kw) == BAD, kw
    assert step(N=2 ** 30, D=2 ** 20) == UNSUPPORTED
    assert step(N=0, x=None, la=None, s=None, o=None) == 0


def test_launches_of_too_many_threads_are_refused(L):
    """The limits lie where a launch of 32-bit threads ends, and no lower."""
    rows = lambda tokens, **kw: L.kda_cache4_append(cache(heads=8, d=128, **kw), tokens, kda.KDA_BF16, FAKE, FAKE, None, None)
    assert rows(2 ** 25 - 32) == BAD and rows(2 ** 25) == UNSUPPORTED          # no slots, too many rows
    call = lambda **kw: L.kda_cache4_attention(cache(), problem(**kw), None, FAKE, FAKE, None, None, FAKE, None, 0, None)
    assert call(n_seq=2 ** 22, tokens=2 ** 22) == BAD and call(n_seq=2 ** 23, tokens=2 ** 23) == UNSUPPORTED
    fwd = lambda **kw: L.kda_recurrence_prefill(rec(**kw), None, FAKE, None, None, None, FAKE, None, FAKE, 1 << 50, None)
    assert fwd(batch=2 ** 22 - 1, seqlen=100, width=100) == BAD and fwd(batch=2 ** 22, seqlen=100, width=100) == UNSUPPORTED
    step = lambda n: L.kda_recurrence_step(n, 1, kda.KDA_F32, -0.5, None, FAKE, None, FAKE, FAKE, None)
    assert step(2 ** 33) == BAD and step(2 ** 33 + 1) == UNSUPPORTED
    # the attention does not write over its queries
    assert L.kda_cache4_attention(cache(), problem(), FAKE, FAKE, FAKE, None, None, FAKE, FAKE, 1 << 40, None) == BAD


def test_binding_refusals():
    """What the Python calls refuse, on tensors that never reach a device."""
    torch = pytest.importorskip("torch")
    i32, z = torch.int32, torch.zeros
    plan = lambda **kw: kda.plan_requests(*[{**dict(a=z(3, dtype=i32), b=z(3, dtype=i32), t=z(3, 4, dtype=i32),
                                                    f=z(5, dtype=i32), p=64, n=3), **kw}[k] for k in "abtfpn"])
    for kw, err in ((dict(b=z(2, dtype=i32)), ValueError), (dict(a=z(3)), TypeError), (dict(t=z(3, dtype=i32)), ValueError),
                    (dict(t=z(2, 4, dtype=i32)), ValueError), (dict(f=z(5)), TypeError), (dict(p=24), ValueError),
                    (dict(n=-1), ValueError), (dict(), ValueError)):      # the last: not on a GPU
        with pytest.raises(err):
            plan(**kw)
    with pytest.raises(ValueError):
        kda.Cache4.empty(4, 24, 2, 128, device="cpu")
    with pytest.raises(ValueError):
        kda.Cache4.empty(4, 64, 2, 96, device="cpu")
    c = kda.Cache4.empty(4, 64, 2, 128, device="cpu")
    with pytest.raises(ValueError):
        kda.Cache4(c.k, c.k_scale[:2], c.v, c.v_scale)
    with pytest.raises(TypeError):
        kda.Cache4(c.k.float(), c.k_scale, c.v, c.v_scale)
    k, slots = z(5, 2, 128), z(5, dtype=torch.int64)
    for kw, err in ((dict(k=k.half()), TypeError), (dict(v=z(4, 2, 128)), ValueError), (dict(v=k.bfloat16()), TypeError),
                    (dict(s=z(5, dtype=i32)), TypeError), (dict(s=z(5, 1, dtype=torch.int64)), ValueError), (dict(), ValueError)):
        with pytest.raises(err):
            kda.cache4_append(c, *[{**dict(k=k, v=k, s=slots), **kw}[n] for n in "kvs"])
    with pytest.raises(TypeError):
        kda.cache4_read(c, slots, torch.float16)
    q, table, total = z(3, 8, 128), z(3, 4, dtype=i32), z(3, dtype=i32)
    for kw, err in ((dict(q=z(3, 7, 128)), ValueError), (dict(q=z(3, 8, 64)), ValueError), (dict(table=z(2, 4, dtype=i32)), ValueError),
                    (dict(total=z(3)), TypeError), (dict(cu=z(3, dtype=i32)), ValueError), (dict(cu=z(4)), TypeError),
                    (dict(g=z(3, 8, 128).bfloat16()), TypeError), (dict(out=z(2, 8, 128)), ValueError), (dict(q=q.half()), TypeError)):
        a = {**dict(q=q, table=table, total=total, cu=None, g=None, out=None), **kw}
        with pytest.raises(err):
            kda.cache4_attention(a["q"], c, a["table"], a["total"], cu_seqlens=a["cu"], g=a["g"], out=a["out"])
    x, s = z(2, 5, 6), z(2, 6)
    for kw, err in ((dict(x=z(2, 5)), ValueError), (dict(la=z(2, 5, 7)), ValueError), (dict(la=x.bfloat16()), TypeError),
                    (dict(g=x.bfloat16()), TypeError), (dict(s=z(1, 6)), ValueError), (dict(cu=z(3, dtype=i32)), ValueError),
                    (dict(), ValueError)):
        a = {**dict(x=x, la=x, g=None, s=s, cu=None), **kw}
        for f in (kda.recurrence_prefill, kda.recurrence_prefill_for_backward, kda.recurrence_autograd):
            with pytest.raises(err):
                f(a["x"], a["la"], -0.5, g=a["g"], state_in=a["s"], cu_seqlens=a["cu"])
    with pytest.raises(ValueError):
        kda.recurrence_step(s, s, z(2, 5), -0.5)
    # strides
    turned = z(6, 2).t()
    for f in (lambda: kda.recurrence_step(turned, turned, turned, -0.5),
              lambda: kda.recurrence_prefill(z(1, 1, 6).expand(2, 5, 6), x, -0.5),
              lambda: kda.cache4_append(c, z(2, 5, 128).transpose(0, 1), k, slots),
              lambda: kda.cache4_attention(z(8, 3, 128).transpose(0, 1), c, table, total),
              lambda: kda.plan_requests(z(6, dtype=i32)[::2], z(3, dtype=i32), z(3, 4, dtype=i32), z(5, dtype=i32), 64, 3)):
        with pytest.raises(ValueError, match="contiguous"):
            f()


def attention_without_queries(c, p):
    """What the call says to a problem before it looks at the queries, which are missing."""
    L = hybrid._hlib()
    return L.kda_cache4_attention(c, p, None, FAKE, FAKE, FAKE, None, FAKE, FAKE, 1 << 50, None)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_attention_refuses_positions_that_tiles_would_carry_past_32_bits(L, page):
    """Positions go up in tiles and units of up to 128 tokens: the last one has to stay below 2^31."""
    room = 2 ** 31 - 1 - 256
    for most, want in ((room // page, BAD), (room // page + 1, UNSUPPORTED), ((2 ** 31 - 1) // page, UNSUPPORTED)):
        p = problem(max_pages=most, tokens=9, max_q=9, max_len=2 ** 31)
        assert attention_without_queries(cache(page_size=page), p) == want, (page, most)
        assert (L.kda_cache4_attention_workspace_size(cache(page_size=page), p) > 0) == (want == BAD)


def test_attention_of_too_many_heads_is_refused(L):
    """A workgroup of 256 threads for every key/value head and share of the work: 2^32 threads are too many."""
    one = dict(n_seq=1, tokens=1, max_pages=1, max_len=0)
    for heads, want in ((2 ** 24 - 1, BAD), (2 ** 24, UNSUPPORTED), (2 ** 28, UNSUPPORTED)):
        c, p = cache(pages=1, page_size=16, d=64, heads=heads), problem(heads=heads, **one)
        assert attention_without_queries(c, p) == want, heads
        assert (L.kda_cache4_attention_workspace_size(c, p) > 0) == (want == BAD)


def test_attention_units_are_dealt_out_below_2_to_the_31(L):
    """Sequences whose units come close to 2^31 have a workgroup a block: a share's end is formed in 32 bits."""
    units = lambda n: (2 ** 31 - 1) // (n + n // 16)          # of n sequences' slots: one page each, 5 for a block
    size = lambda n, pages: L.kda_cache4_attention_workspace_size(
        cache(page_size=128, heads=1, d=64), problem(n_seq=n, tokens=n, heads=1, max_pages=pages, max_len=2 ** 40))
    assert size(128, units(128) - 5 - 16) > 0 and size(128, units(128) - 5) == 0


def test_attention_refuses_scales_whose_exponents_end(L):
    """Scores are formed in powers of two: scale * log2(e) has to be a normal number, or 0."""
    for scale, want in ((0.0, BAD), (-0.0, BAD), (1e-37, BAD), (-2.3e38, BAD), (2.0 ** 127, BAD), (2.0 ** -126, BAD),
                        (2.4e38, UNSUPPORTED), (-3.4e38, UNSUPPORTED), (1e-39, UNSUPPORTED), (-1e-45, UNSUPPORTED)):
        assert attention_without_queries(cache(), problem(tokens=9, scale=scale)) == want, scale


def test_gradients_are_aligned_before_the_call():
    torch = pytest.importorskip("torch")
    room = torch.arange(40, dtype=torch.float32)
    for d in (None, room[:12], room[4:16].view(3, 4), room[3:15].view(3, 4), room[:12].view(3, 4).t(), room[:1].expand(3, 4),
              room.bfloat16()[1:5]):
        got = hybrid._gradient(d)
        assert got is None if d is None else got.is_contiguous() and got.data_ptr() % 16 == 0 and torch.equal(got, d)
    assert hybrid._gradient(room) is room               # nothing is copied without need
