"""Attention over the 4-bit cache for groups of sequences that share their first
tokens, on an MI355X against a plain 64-bit form.

Tolerance per output: that of tests/test_gpu_cache4_attention.py (a score's sum
of d products, twice; the probabilities' rounding; n u32 for sums over the
tokens; 16 u32 for exponential, reciprocal and gate; the output's rounding), and
8 u32 more, as the two parts of a row are joined with two more exponentials, two
products and a sum each for the values and the weights."""
import math

import pytest

import _hybrid_ref as ref

torch = pytest.importorskip("torch")
import gated_delta_rule_91_amd as kda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def build(offsets, prefix, own, new, heads, kv, d, page, io, seed=0, gate=True):
    """Groups of sequences with `own` tokens each behind their prefix.  What nobody may read stands for NaN and huge
    values: behind each sequence's last token, and in the tables of all but a group's first sequence the whole prefix,
    whose pages are theirs alone here; a prefix may end inside a page."""
    gen = torch.Generator(device="cuda").manual_seed(seed + sum(own) + d + sum(prefix))
    n = len(own)
    first, before = list(range(n)), [0] * n
    for j, p in enumerate(prefix):
        for s in range(offsets[j], offsets[j + 1]):
            first[s], before[s] = offsets[j], p
    total = [b + o for b, o in zip(before, own)]
    pages = sum(-(-t // page) for t in total) + 2
    c = kda.Cache4.empty(pages, page, kv, d)
    for t in (c.k, c.v):
        t.copy_(torch.randint(0, 256, t.shape, generator=gen, device="cuda").to(torch.uint8))
    for t in (c.k_scale, c.v_scale):
        t.copy_(torch.randint(118, 128, t.shape, generator=gen, device="cuda").to(torch.uint8))
    order = torch.randperm(pages, generator=gen, device="cuda").tolist()
    width = max([-(-t // page) for t in total] + [1])
    table, used = [], set()
    for s, t in enumerate(total):
        row = [order.pop() for _ in range(-(-t // page))]
        used |= {row[i // page] * page + i % page for i in range(0 if first[s] == s else before[s], t)}
        table.append(row + [10 ** 6] * (width - len(row)))
    hole = torch.ones(pages * page, dtype=torch.bool)
    hole[list(used)] = False
    hole = hole.view(pages, 1, page, 1).cuda()
    c.k_scale.masked_fill_(hole, 255)
    c.v_scale.masked_fill_(hole, 254)
    T = sum(new)
    q = torch.randn(T, heads, d, generator=gen, device="cuda").to(DT[io])
    g = torch.randn(T, heads, d, generator=gen, device="cuda").to(DT[io]) if gate else None
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    return dict(c=c, q=q, g=g, table=table, total=total, cu=cu, offsets=offsets, prefix=prefix, first=first, before=before)


def attention(b, scale):
    """(out, sum p |v|, bound on the scores' size) in 64 bits; rows of no sequence are NaN."""
    c, q = b["c"], b["q"].cpu().double()
    T, Hq, d = q.shape
    H, page = c.heads, c.page_size
    k, v = (ref.values(getattr(c, n).cpu(), getattr(c, n + "_scale").cpu()).transpose(1, 2).reshape(-1, H, d) for n in ("k", "v"))
    out = torch.full((T, Hq, d), math.nan, dtype=torch.float64)
    mag, size = torch.zeros_like(out), 0.0
    for s, total in enumerate(b["total"]):
        r0, r1 = b["cu"][s], b["cu"][s + 1]
        rows = [b["table"][b["first"][s]][t // page] if t < b["before"][s] else b["table"][s][t // page] for t in range(total)]
        ok = torch.tensor([0 <= r < c.pages for r in rows], dtype=torch.bool)
        at = torch.tensor([r * page + t % page if 0 <= r < c.pages else 0 for t, r in enumerate(rows)], dtype=torch.long)
        for row in range(r0, r1):
            end = min(max(total - (r1 - r0) + (row - r0) + 1, 0), total)
            seen = at[:end][ok[:end]]
            for h in range(Hq):
                kv = h // (Hq // H)
                if not len(seen):
                    out[row, h] = 0
                    continue
                w = torch.softmax(k[seen, kv] @ q[row, h] * scale, 0)
                out[row, h], mag[row, h] = w @ v[seen, kv], w @ v[seen, kv].abs()
                size = max(size, float((k[seen, kv].abs() @ q[row, h].abs()).max()) * abs(scale))
    if b["g"] is not None:
        sig = torch.sigmoid(b["g"].cpu().double())
        out, mag = out * sig, mag * sig
    return out, mag, size


def check(b, io, scale=None, decode=False, **kw):
    c, q = b["c"], b["q"]
    scale = 1 / math.sqrt(c.d) if scale is None else scale
    room = torch.full((q.shape[0] + 4, *q.shape[1:]), 77.0, dtype=q.dtype, device="cuda")
    out = room[2:-2]                                      # nothing is written around it
    got = kda.cache4_shared_attention(q, c, i32(b["table"]).reshape(len(b["total"]), -1), i32(b["total"]), i32(b["prefix"]), i32(b["offsets"]),
                                      cu_seqlens=None if decode else i32(b["cu"]), g=b["g"], scale=scale, out=out, **kw)
    torch.cuda.synchronize()
    assert got is out and (room[:2] == 77.0).all() and (room[-2:] == 77.0).all()
    want, mag, size = attention(b, scale)
    got = out.cpu().double()
    none = torch.isnan(want).all(-1).all(-1)              # rows of no sequence stay as they were
    assert (got[none] == 77.0).all()
    want, got, mag = want[~none], got[~none], mag[~none]
    u32, n = 2.0 ** -24, max(b["total"] + [1])
    tol = (2 * (c.d + 8) * u32 * size + n * u32 + 24 * u32 + (U[io] if io == "bf16" else u32)) * mag + U[io] * want.abs() + 1e-30
    worst = float(((got - want).abs() / tol).max()) if got.numel() else 0.0
    assert worst <= 1, worst
    return out


CASES = [([0, 2], [64], [1, 1]), ([0, 3], [100], [1, 40, 17]), ([0, 5], [130], [3, 1, 200, 33, 16]), ([0, 2, 5], [33, 257], [5, 9, 1, 70, 2]),
         ([1, 3, 6], [15, 90], [20, 4, 1, 60, 5, 2, 31]), ([0, 1, 3], [70, 40], [6, 3, 8]), ([0, 4], [1], [1, 2, 3, 4]), ([0, 9], [700], [2] * 9)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv,d,page", [(8, 2, 128, 64), (3, 3, 64, 16), (12, 1, 64, 32), (16, 1, 128, 16), (34, 2, 128, 256)])
@pytest.mark.parametrize("offsets,prefix,own", CASES)
def test_decode(offsets, prefix, own, heads, kv, d, page, io):
    b = build(offsets, prefix, own, [1] * len(own), heads, kv, d, page, io)
    check(b, io, decode=True)
    check(dict(b, g=None), io, max_prefix=max(prefix), max_own=max(own))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv,d,page", [(4, 2, 128, 64), (6, 6, 64, 16), (20, 1, 64, 16), (8, 1, 128, 32)])
@pytest.mark.parametrize("offsets,prefix,own,new", [([0, 2], [50], [30, 7], [30, 7]), ([0, 3], [100], [3, 60, 17], [1, 40, 17]),
                                                    ([1, 3, 5], [77, 33], [20, 9, 31, 1, 150, 4], [2, 9, 5, 1, 140, 4]), ([0, 4], [200], [9, 4, 80, 30], [0, 3, 70, 0])])
def test_many_queries(offsets, prefix, own, new, heads, kv, d, page, io):
    b = build(offsets, prefix, own, new, heads, kv, d, page, io)
    check(b, io, max_q=max(new), max_prefix=max(prefix), max_own=max(own))
    check(dict(b, g=None), io, scale=-0.3)


def test_many_sequences_and_a_long_prefix():
    """Enough rows for the form in which each wave has its own, and parts to join."""
    n = 70
    b = build([0, n], [1500], [1 + (5 * i) % 23 for i in range(n)], [1] * n, 8, 2, 64, 16, "bf16")
    check(b, "bf16", decode=True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,heads,kv,d", [(64, 16, 2, 64), (40, 16, 1, 128), (20, 16, 1, 64)])
def test_rows_in_many_parts(n, heads, kv, d, io):
    """More than 512 rows, and fewer, of a long prefix that many workgroups share."""
    check(build([0, n], [2900], [1 + s % 5 for s in range(n)], [1] * n, heads, kv, d, 16, io), io, decode=True)


@pytest.mark.parametrize("heads", [2, 17])
def test_more_sequences_than_are_dealt_out(heads):
    """Blocks past 4096 are a workgroup's, or a wave's, each."""
    n = 4400
    offsets = list(range(0, n + 1, 2))
    check(build(offsets, [5 + j % 30 for j in range(n // 2)], [1 + s % 7 for s in range(n)], [1] * n, heads, 1, 64, 16, "bf16", gate=False), "bf16",
          decode=True)


def test_sequences_without_queries():
    check(build([0, 4, 6], [40, 21], [9, 20, 3, 5, 2, 2], [0, 20, 3, 0, 0, 0], 8, 2, 128, 16, "bf16"), "bf16")


def test_more_groups_than_sequences_and_none():
    """Empty groups, groups that hold nothing but queries of nobody, and no group at all."""
    b = build([0, 0, 2, 2, 2, 3], [5, 40, 7, 9, 30], [4, 5, 6], [1, 1, 1], 4, 2, 64, 16, "f32")
    check(b, "f32", decode=True)
    alone = kda.cache4_attention(b["q"], b["c"], i32(b["table"]), i32([4, 5, 6]), g=b["g"])
    none = kda.cache4_shared_attention(b["q"], b["c"], i32(b["table"]), i32([4, 5, 6]), i32([]), i32([0]), g=b["g"])
    torch.cuda.synchronize()
    assert torch.equal(alone.nan_to_num(), none.nan_to_num())


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_a_prefix_that_not_all_queries_see(io):
    """As much of it is shared as lies before every query: the tables name the same pages, so the rest is read there."""
    b = build([0, 3], [0], [200, 200, 200], [1, 1, 1], 8, 2, 128, 16, io)
    b["table"] = [b["table"][0]] * 3
    b["total"] = [200, 37, 100]
    for p in (36, 37, 50, 200, 10 ** 6, -5, 2 ** 31 - 1):
        check(dict(b, prefix=[p]), io, decode=True)
    b["total"] = [200, 0, 100]                            # one that has nothing to see
    out = check(dict(b, prefix=[64]), io, decode=True)
    assert (out[1] == 0).all()


def test_bad_pages_are_left_out():
    b = build([0, 3], [100], [20, 30, 9], [1, 1, 1], 8, 2, 64, 16, "f32")
    b["table"][0][2], b["table"][0][5], b["table"][1][7] = -1, 10 ** 9, b["c"].pages
    b["table"][2] = [-1] * len(b["table"][2])             # all of its own tokens
    check(b, "f32", decode=True)


@pytest.mark.parametrize("offsets,prefix", [([5, 1], [10]), ([-7, 100], [40]), ([2, 2 ** 31 - 1], [-1]), ([3, 2, 1, 0], [9, 9, 9])])
def test_bad_offsets_stay_inside(offsets, prefix):
    """Rows may be anything then, and nothing around them changes."""
    b = build([0, 4], [50], [20, 30, 9, 4], [1] * 4, 4, 2, 64, 16, "f32")
    room = torch.full((8, 4, 64), 77.0, device="cuda")
    kda.cache4_shared_attention(b["q"], b["c"], i32(b["table"]), i32(b["total"]), i32(prefix), i32(offsets), out=room[2:-2])
    torch.cuda.synchronize()
    assert (room[:2] == 77.0).all() and (room[-2:] == 77.0).all()


def test_hints_change_nothing_but_the_split():
    b = build([0, 3, 4], [300, 20], [50, 3, 9, 80], [1, 1, 1, 1], 8, 2, 128, 16, "f32")
    for max_q in (1, 100, 10 ** 9):
        for most in (0, 60, 10 ** 9):
            check(b, "f32", max_q=max_q, max_prefix=most, max_own=most)


def test_nan_reaches_its_queries_only():
    """A value that is no number: in a prefix for its group's rows, elsewhere for its own."""
    b = build([0, 2, 4], [50, 40], [9, 8, 7, 6], [1] * 4, 4, 2, 64, 16, "f32")
    c, t = b["c"], b["table"]
    c.v_scale[t[0][1], 0, 3, 1] = 255                     # token 19 of the first group, head 0, channels 32..63
    c.k_scale[t[3][2], 1, 10, 0] = 255                    # token 42 of the last sequence, head 1
    out = kda.cache4_shared_attention(b["q"], c, i32(t), i32(b["total"]), i32(b["prefix"]), i32(b["offsets"]), g=b["g"])
    torch.cuda.synchronize()
    want = torch.zeros(4, 4, 64, dtype=torch.bool)
    want[:2, :2, 32:] = True
    want[3, 2:] = True
    assert torch.equal(torch.isnan(out.cpu()), want)


def test_given_workspace_and_what_it_held():
    b = build([1, 4, 6], [200, 77], [9, 50, 3, 20, 4, 31, 6], [1] * 7, 8, 2, 128, 16, "bf16")
    args = (b["q"], b["c"], i32(b["table"]), i32(b["total"]), i32(b["prefix"]), i32(b["offsets"]))
    want = kda.cache4_shared_attention(*args, g=b["g"])
    size = kda.cache4_shared_attention_workspace_size(*args)
    for fill in (0, 1, 127, 255):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            got = kda.cache4_shared_attention(*args, g=b["g"], workspace=ws)
            torch.cuda.synchronize()
            assert torch.equal(got, want)
    with pytest.raises(kda.KdaError) as e:
        kda.cache4_shared_attention(*args, g=b["g"], workspace=ws[:-256])
    assert e.value.code == 3
