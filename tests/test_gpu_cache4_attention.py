"""Attention over the 4-bit cache on an MI355X against a plain 64-bit form.

Tolerance per output, from the roundings that the kernel may make (u: half a
step, 2^-8 bf16, 2^-24 fp32; |V| weighted by the probabilities = mag):
  scores: a sum of d products in fp32, off by at most (d + 8) u32 S with S the
  largest sum |q||k| scale; exp of it shifts every probability by as much
  again, relatively, and the sum that divides them too: 2 (d + 8) u32 S mag;
  probabilities round to bf16 (bf16) or to three bf16 parts (fp32: below u32),
  sums over the tokens in fp32: n u32 mag;  exp2 and reciprocal, gate: 16 u32;
  the output rounds once: u |out|."""
import math

import pytest

import _hybrid_ref as ref

torch = pytest.importorskip("torch")
import gated_delta_rule_91_amd as kda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def build(total, new, heads, kv, d, page, io, seed=0, gate=True, spare=2):
    """Tensors of a cache whose pages lie anywhere, garbage behind every sequence's last token."""
    gen = torch.Generator(device="cuda").manual_seed(seed + sum(total) + d)
    n = len(total)
    width = max([-(-t // page) for t in total] + [1])
    pages = sum(-(-t // page) for t in total) + spare
    c = kda.Cache4.empty(pages, page, kv, d)
    for t in (c.k, c.v):
        t.copy_(torch.randint(0, 256, t.shape, generator=gen, device="cuda").to(torch.uint8))
    for t in (c.k_scale, c.v_scale):
        t.copy_(torch.randint(118, 128, t.shape, generator=gen, device="cuda").to(torch.uint8))
    order = torch.randperm(pages, generator=gen, device="cuda").tolist()
    table, used = [], set()
    for t in total:
        row = [order.pop() for _ in range(-(-t // page))]
        used |= {p * page + i for j, p in enumerate(row) for i in range(min(page, t - j * page))}
        table.append(row + [10 ** 6] * (width - len(row)))       # pages that do not exist behind the last
    # what no sequence holds stands for NaN and huge values
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
    return c, q, g, table, cu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check(c, q, g, table, total, cu, io, scale=None, decode=False, **kw):
    scale = 1 / math.sqrt(c.d) if scale is None else scale
    room = torch.full((q.shape[0] + 4, *q.shape[1:]), 77.0, dtype=q.dtype, device="cuda")
    out = room[2:-2]                                      # nothing is written around it
    got = kda.cache4_attention(q, c, i32(table).reshape(len(total), -1), i32(total), cu_seqlens=None if decode else i32(cu), g=g,
                               scale=scale, out=out, **kw)
    torch.cuda.synchronize()
    assert got is out
    host = {n: getattr(c, n).cpu() for n in ("k", "k_scale", "v", "v_scale")}
    want, mag, size = ref.attention(q.cpu(), host, table, total, cu, scale, None if g is None else g.cpu())
    assert (room[:2] == 77.0).all() and (room[-2:] == 77.0).all()
    got = out.cpu().double()
    none = torch.isnan(want).all(-1).all(-1)              # rows of no sequence stay as they were
    assert (got[none] == 77.0).all()
    want, got, mag = want[~none], got[~none], mag[~none]
    u32 = 2.0 ** -24
    n = max(list(total) + [1])
    tol = (2 * (c.d + 8) * u32 * size + n * u32 + 16 * u32 + (U[io] if io == "bf16" else u32)) * mag + U[io] * want.abs() + 1e-30
    worst = float(((got - want).abs() / tol).max()) if got.numel() else 0.0
    assert worst <= 1, worst
    return out


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv,d,page", [(8, 2, 128, 64), (3, 3, 64, 16), (12, 1, 64, 32), (16, 1, 128, 16),
                                             (34, 2, 128, 256), (40, 1, 64, 64)])
@pytest.mark.parametrize("total", [[1], [15, 16, 17, 1, 33], [600, 31, 257], [2100, 3]])
def test_decode(total, heads, kv, d, page, io):
    c, q, g, table, cu = build(total, [1] * len(total), heads, kv, d, page, io)
    check(c, q, g, table, total, cu, io, decode=True)
    check(c, q, None, table, total, cu, io, max_len=max(total))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv,d,page", [(4, 2, 128, 64), (3, 1, 64, 16), (6, 6, 128, 32), (20, 1, 64, 16)])
@pytest.mark.parametrize("total,new", [([40], [40]), ([70, 5, 130], [3, 5, 129]), ([200, 33, 64, 1], [17, 1, 64, 1]),
                                       ([300], [2])])
def test_many_queries(total, new, heads, kv, d, page, io):
    c, q, g, table, cu = build(total, new, heads, kv, d, page, io)
    check(c, q, g, table, total, cu, io, max_q=max(new), max_len=max(total))
    check(c, q, None, table, total, cu, io, scale=-0.3)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv,d", [(8, 2, 128), (8, 1, 64), (3, 1, 128)])
@pytest.mark.parametrize("new", [4, 5, 8, 9, 12, 13, 24, 25])
def test_few_queries(new, heads, kv, d, io):
    """Around the sizes of a row block and the rule that chooses how its rows are shared."""
    total, many = [150, new, 1100, 40], [new, new, new, 1]
    c, q, g, table, cu = build(total, many, heads, kv, d, 32, io)
    check(c, q, g, table, total, cu, io, max_q=new, max_len=max(total))


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_rows_that_see_nothing_and_rows_of_no_sequence(io):
    total, new = [4, 0, 20, 3], [6, 2, 0, 1]              # more queries than tokens: the first see nothing
    c, q, g, table, cu = build(total, new, 8, 2, 128, 16, io)
    q = torch.cat([q, q[:3]]).contiguous()
    g = torch.cat([g, g[:3]]).contiguous()
    out = check(c, q, g, table, total, cu, io)
    assert (out[:2] == 0).all() and (out[6:8] == 0).all()
    total = [0, 5]
    c, q, g, table, cu = build(total, [1, 1], 8, 2, 64, 16, io)
    check(c, q, g, table, total, cu, io, decode=True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_bad_pages_are_left_out(io):
    total, new = [100, 90, 64], [1, 5, 3]
    c, q, g, table, cu = build(total, new, 8, 2, 128, 16, io)
    table[0][2], table[0][5], table[1][0], table[1][5] = -1, 10 ** 9, -2 ** 31, c.pages
    table[2] = [-1] * len(table[2])                       # nothing at all
    out = check(c, q, g, table, total, cu, io)
    assert (out[6:] == 0).all()
    # longer than the table: its rows are the end.  What lay behind the last tokens counts now, so it is no NaN here
    c.k_scale.masked_fill_(c.k_scale == 255, 120)
    c.v_scale.masked_fill_(c.v_scale == 254, 120)
    check(c, q, g, table, [10 ** 6, 95, 2 ** 31 - 1], cu, io)


def test_hints_change_nothing_but_the_split():
    total, new = [1500, 700, 3], [1, 1, 1]
    c, q, g, table, cu = build(total, new, 8, 2, 128, 16, "f32")
    for max_q in (1, 2, 100, 10 ** 9):
        for max_len in (0, 1, 700, 1500, 10 ** 9):
            check(c, q, g, table, total, cu, "f32", max_q=max_q, max_len=max_len)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_extreme_scores(io):
    """Scores far apart and all alike: the running maximum carries them."""
    total, new = [300, 40], [2, 1]
    c, q, g, table, cu = build(total, new, 4, 2, 64, 16, io)
    check(c, q, g, table, total, cu, io, scale=0.0)
    # size of the scores some hundreds: the tolerance grows with it; most weights vanish
    check(c, q, g, table, total, cu, io, scale=2.0)


def test_nan_in_the_cache_reaches_only_its_queries():
    total, new = [50, 50], [1, 1]
    c, q, g, table, cu = build(total, new, 4, 2, 64, 16, "f32")
    c.v_scale[table[0][1], 0, 3, 1] = 255                 # token 19 of sequence 0, head 0, channels 32..63
    c.k_scale[table[1][0], 1, 2, 0] = 255                 # token 2 of sequence 1, head 1
    out = kda.cache4_attention(q, c, i32(table), i32(total), g=g)
    torch.cuda.synchronize()
    bad = torch.isnan(out.cpu())
    want = torch.zeros_like(bad)
    want[0, :2, 32:] = True
    want[1, 2:] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d,heads", [(64, 20), (128, 3)])
def test_nan_that_some_queries_do_not_see(d, heads, io):
    """Values that are NaN or Inf reach the queries behind them and no others, wherever the block table's stretches end."""
    total, new, page = [1200], [200], 16
    c, q, g, table, cu = build(total, new, heads, 1, d, page, io)
    for t, scale in ((1010, 255), (1100, 255), (1153, 254)):
        c.v_scale[table[0][t // page], 0, t % page, 0] = scale
        c.v[table[0][t // page], 0, t % page] = 0x77      # 6 and 6: 6 times 2^127 is Inf
    out = kda.cache4_attention(q, c, i32(table), i32(total), cu_seqlens=i32(cu), g=g, max_q=200, max_len=1200)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(out.cpu().float())
    want = torch.zeros_like(bad)
    want[10:, :, :32] = True                              # query i is at position 1000 + i
    assert torch.equal(bad, want)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("heads,d", [(2, 64), (4, 128)])
def test_nan_that_some_of_few_queries_do_not_see(heads, d, io):
    """The same for as few rows as waves share: 6 queries of 2 or 4 heads."""
    total, new = [40, 37], [6, 1]
    c, q, g, table, cu = build(total, new, heads, 1, d, 16, io)
    c.v_scale[table[0][2], 0, 5, 1] = 255                 # token 37 of sequence 0, channels 32..63
    out = kda.cache4_attention(q, c, i32(table), i32(total), cu_seqlens=i32(cu), g=g, max_q=6)
    torch.cuda.synchronize()
    bad = torch.isnan(out.cpu().float())
    want = torch.zeros_like(bad)
    want[3:6, :, 32:64] = True                            # query i is at position 34 + i
    assert torch.equal(bad, want)


def test_given_workspace():
    total = [900, 40]
    c, q, g, table, cu = build(total, [1, 1], 8, 2, 128, 16, "bf16")
    t, n = i32(table), i32(total)
    want = kda.cache4_attention(q, c, t, n, g=g)
    size = kda.cache4_attention_workspace_size(q, c, t, n)
    assert size > 0
    for fill in (0, 255, 127):                            # whatever it holds before
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            got = kda.cache4_attention(q, c, t, n, g=g, workspace=ws)
            torch.cuda.synchronize()
            assert torch.equal(got, want)
    with pytest.raises(kda.KdaError) as e:
        kda.cache4_attention(q, c, t, n, g=g, workspace=ws[:-256])
    assert e.value.code == 3
    with pytest.raises(ValueError):
        kda.cache4_attention(q.transpose(0, 1).contiguous().transpose(0, 1), c, t, n)      # strides


def test_what_a_workspace_held_does_not_count():
    """Sequences without queries or tokens leave nothing in it."""
    total, new = [2000, 70, 0, 40, 3000], [1, 0, 2, 9, 0]
    c, q, g, table, cu = build(total, new, 8, 2, 128, 16, "bf16")
    t, n, cut = i32(table), i32(total), i32(cu)
    want = kda.cache4_attention(q, c, t, n, cut, g=g, max_q=9)
    size = kda.cache4_attention_workspace_size(q, c, t, n, cut, max_q=9)
    assert size > 0
    for fill in (0, 1, 127, 255):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        got = kda.cache4_attention(q, c, t, n, cut, g=g, max_q=9, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_many_blocks_without_dealing_out():
    """More row blocks than prefix sums are kept for: a workgroup each."""
    n = 4200
    total = [1 + (7 * i) % 40 for i in range(n)]
    c, q, g, table, cu = build(total, [1] * n, 2, 1, 64, 16, "bf16", gate=False)
    check(c, q, None, table, total, cu, "bf16", decode=True)


def test_offsets_past_32_bits():
    """A cache of over 4 GiB a part: its last pages are read and written in place."""
    pages, page, heads, d = 270000, 256, 1, 128           # 4.4e9 bytes of keys
    c = kda.Cache4.empty(pages, page, heads, d)
    T = 300
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(T, heads, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    slots = torch.cat([torch.arange(256), torch.arange(44) + 256 * (pages - 1)]).cuda()
    kda.cache4_append(c, k, v, slots)
    rk, rv = kda.cache4_read(c, slots, torch.bfloat16)
    q = torch.randn(1, 4, d, generator=gen, device="cuda").bfloat16()
    out = kda.cache4_attention(q, c, i32([[0, pages - 1]]), i32([T]))
    torch.cuda.synchronize()
    k8, v8 = rk.cpu().double()[:, 0], rv.cpu().double()[:, 0]
    codes, sc = ref.quantized(k.cpu())
    assert torch.equal(k8, ref.values(ref.packed(codes), sc)[:, 0])
    s = q.cpu().double()[0] @ k8.T / math.sqrt(d)
    p = torch.softmax(s, -1)
    want, mag = p @ v8, p @ v8.abs()
    tol = (2.0 ** -8 + 2.0 ** -13) * mag + 2.0 ** -8 * want.abs()
    assert ((out.cpu().double()[0] - want).abs() <= tol).all()
    del c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("new", [[2, 1], [200, 30]])
def test_a_scale_of_zero_weighs_all_alike(new, io):
    """However large the products are that it takes away."""
    total = [300, 40]
    c, q, g, table, cu = build(total, new, 4, 2, 64, 16, io)
    check(c, (q.float() * 1e35).to(q.dtype), g, table, total, cu, io, scale=0.0, max_q=max(new))
    check(c, (q.float() * 1e35).to(q.dtype), g, table, total, cu, io, scale=-0.0, max_q=max(new))


@pytest.mark.parametrize("io,total,new", [("bf16", [5300, 0, 2000, 40, 1500], [4800, 3, 1900, 0, 1500]),
                                          ("f32", [2600, 0, 1000, 40, 800], [2400, 3, 950, 0, 800])])
@pytest.mark.parametrize("heads,kv,d", [(64, 1, 64), (64, 1, 128)])
def test_many_blocks_of_many_rows(heads, kv, d, io, total, new):
    """Prompts of more row blocks than prefix sums are kept for, with offsets; some rows against the 64-bit form."""
    rows = {"bf16": 128, "f32": 64}[io]
    assert sum(new) * heads // kv // rows + len(new) > 4096
    c, q, g, table, cu = build(total, new, heads, kv, d, 64, io)
    out = torch.full((q.shape[0] + 2, *q.shape[1:]), 77.0, dtype=q.dtype, device="cuda")
    kda.cache4_attention(q, c, i32(table), i32(total), cu_seqlens=i32(cu), g=g, out=out[:-2], max_q=max(new), max_len=max(total))
    assert kda.cache4_attention_workspace_size(q, c, i32(table), i32(total), i32(cu), max_q=max(new)) == 0
    torch.cuda.synchronize()
    assert (out[-2:] == 77.0).all() and (out[cu[1]:cu[2]] == 0).all()
    k, v = (ref.values(getattr(c, n).cpu(), getattr(c, n + "_scale").cpu()) for n in ("k", "v"))
    u32, scale = 2.0 ** -24, 1 / math.sqrt(d)
    for s in (0, 2, 4):
        m = new[s]
        at = torch.tensor([table[s][t // 64] * 64 + t % 64 for t in range(total[s])])
        kk, vv = (x[:, 0].reshape(-1, d)[at] for x in (k, v))
        for i in {0, 1, 63, 64, m // 3, m // 2, m - 2, m - 1}:
            end, row = total[s] - m + i + 1, cu[s] + i
            qq = q[row].cpu().double()
            p = torch.softmax(qq @ kk[:end].T * scale, -1)
            want, mag = p @ vv[:end], p @ vv[:end].abs()
            sig = torch.sigmoid(g[row].cpu().double())
            size = float((qq.abs() @ kk[:end].abs().T).max()) * scale
            tol = (2 * (d + 8) * u32 * size + end * u32 + 16 * u32 + (U[io] if io == "bf16" else u32)) * mag * sig + U[io] * (want * sig).abs() + 1e-30
            assert ((out[row].cpu().double() - want * sig).abs() <= tol).all(), (s, i)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_many_ragged_sequences_without_dealing_out(io):
    """The offsets of over 4096 sequences, searched in memory: some without queries, some of two blocks."""
    n = 4300
    new = [(5 * i) % 3 if i % 97 else 12 for i in range(n)]
    total = [m + (7 * i) % 30 for i, m in enumerate(new)]
    c, q, g, table, cu = build(total, new, 2, 1, 64, 16, io)
    check(c, q, g, table, total, cu, io, max_q=3)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d,heads", [(64, 4), (128, 2)])
@pytest.mark.parametrize("others", [0, 69, 600])
def test_joins_of_more_parts_than_lanes(others, d, heads, io):
    """A context whose parts a wave joins in more than one turn: alone, and beside few and many short ones."""
    total, new = [45000 if others < 600 else 60000] + [1] * others, [2] + [1] * others
    c, q, g, table, cu = build(total, new, heads, 1, d, 256, io)
    check(c, q, g, table, total, cu, io, max_q=2, max_len=max(total))
    check(c, q, g, table, total, cu, io, max_q=2, max_len=max(total), scale=3.0)
