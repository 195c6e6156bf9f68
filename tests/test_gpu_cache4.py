"""The 4-bit cache on an MI355X: append and read against a plain form that
rounds one value at a time in 64 bits.  Codes and scales are whole numbers and
the values they stand for are exact, so everything has to be equal."""
import math

import pytest

import _hybrid_ref as ref

torch = pytest.importorskip("torch")
import gated_delta_rule_91_amd as kda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def cache_of(pages, page, heads, d, fill=0xA5):
    c = kda.Cache4.empty(pages, page, heads, d)
    for t in (c.k, c.k_scale, c.v, c.v_scale):
        t.fill_(fill)
    return c


def check(c, k, v, slots):
    """Append, compare the whole cache (untouched rows too), read back."""
    before = [t.cpu() for t in (c.k, c.k_scale, c.v, c.v_scale)]
    kda.cache4_append(c, k, v, slots)
    rk, rv = kda.cache4_read(c, slots, k.dtype)
    torch.cuda.synchronize()
    page = c.page_size
    got = [t.cpu() for t in (c.k, c.k_scale, c.v, c.v_scale)]
    for x, data, scale, back in ((k, 0, 1, rk), (v, 2, 3, rv)):
        codes, sc = ref.quantized(x.cpu())
        codes = ref.packed(codes)
        for t, s in enumerate(slots.tolist()):
            if 0 <= s < c.pages * page:
                before[data][s // page, :, s % page] = codes[t]
                before[scale][s // page, :, s % page] = sc[t]
        want = ref.values(codes, sc)
        inside = ((slots >= 0) & (slots < c.pages * page)).cpu()
        want[~inside] = 0
        assert torch.equal(torch.nan_to_num(back.cpu().double(), nan=12345.0), torch.nan_to_num(want, nan=12345.0))
    for b, g in zip(before, got):
        assert torch.equal(b, g)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,heads,page", [(1, 1, 16), (5, 3, 16), (67, 2, 64), (300, 1, 256), (33, 8, 32)])
def test_append_and_read(T, heads, page, d, io):
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    c = cache_of(-(-T // page) + 2, page, heads, d)
    k = (torch.randn(T, heads, d, generator=gen, device="cuda") * torch.exp(3 * torch.randn(T, 1, 1, generator=gen, device="cuda"))).to(DT[io])
    v = torch.randn(T, heads, d, generator=gen, device="cuda").to(DT[io])
    slots = torch.randperm(c.pages * page, generator=gen, device="cuda")[:T]
    check(c, k, v, slots)


def test_append_borders():
    """Halves, saturation, zeros, the smallest and the largest scales, Inf and NaN."""
    f = lambda *v: torch.tensor((list(v) + [0.0] * 32)[:32])
    rows = [f(), f(*[-0.0] * 32),
            f(4, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 7),
            f(7.0), f(7.5, 1, 2, 3), f(6.99, .24999, .25001, 4.99, 5.01), f(8, 1, -3, 0.5),
            f(2.0 ** -126, 1e-40, -2.0 ** -127), f(1e-45), f(3.3e38, -2.0 ** 127, 1.9 * 2.0 ** 127), f(2.0 ** 127),
            f(1.75 * 2.0 ** 10), f(1.7500001 * 2.0 ** 10, 1), f(math.inf, 1), f(1, -math.inf), f(math.nan, 2), f(1, 2, 3, math.nan)]
    rows += [f(), f(1.0), f(-1.0)]
    x = torch.stack(rows).reshape(-1, 1, 64).cuda()
    c = cache_of(2, 16, 1, 64)
    check(c, x, x.flip(0).contiguous(), torch.arange(x.shape[0], device="cuda") + 3)
    check(c, x.bfloat16(), x.flip(0).bfloat16().contiguous(), torch.arange(x.shape[0], device="cuda") + 3)


def test_slots_outside_the_cache():
    c = cache_of(3, 16, 2, 128)
    x = torch.randn(6, 2, 128, device="cuda")
    check(c, x, -x, torch.tensor([-1, 48, 2 ** 40, -2 ** 62, 47, 0], device="cuda"))
    empty = torch.empty(0, 2, 128, device="cuda")
    check(c, empty, empty, torch.empty(0, dtype=torch.int64, device="cuda"))
    none = kda.Cache4.empty(0, 16, 2, 128)
    kda.cache4_append(none, x, x, torch.arange(6, device="cuda"))
    k, v = kda.cache4_read(none, torch.arange(6, device="cuda"), torch.bfloat16)
    torch.cuda.synchronize()
    assert not k.any() and not v.any()


def test_every_code_and_scale_reads_as_its_value():
    c = kda.Cache4.empty(17, 16, 1, 64)
    data = torch.arange(256, dtype=torch.uint8).repeat(34)[:17 * 16 * 32].reshape(17, 1, 16, 32)
    scale = torch.arange(17 * 16 * 2).reshape(17, 1, 16, 2).to(torch.uint8)
    for t, x in ((c.k, data), (c.v, data.flip(3).contiguous()), (c.k_scale, scale), (c.v_scale, scale)):
        t.copy_(x)
    k, v = kda.cache4_read(c, torch.arange(17 * 16, device="cuda"), torch.float32)
    torch.cuda.synchronize()
    for got, x in ((k, data), (v, data.flip(3))):
        want = ref.values(x, scale).reshape(-1, 64).float()       # Inf where 4 and 6 times 2^127 pass fp32
        assert torch.equal(torch.nan_to_num(got.cpu().reshape(-1, 64), nan=12345.0, posinf=1, neginf=-1),
                           torch.nan_to_num(want, nan=12345.0, posinf=1, neginf=-1))
