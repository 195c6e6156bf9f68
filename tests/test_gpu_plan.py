"""kda_plan_requests on an MI355X against a plain one-request-at-a-time form:
whole numbers, so everything has to be equal."""
import random

import pytest

import _hybrid_ref as ref

torch = pytest.importorskip("torch")
import gated_delta_rule_91_amd as kda

pytestmark = pytest.mark.gpu


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def check(past, new, table, free, page, tokens):
    n, width = len(past), len(table[0]) if table else 0
    t = ints(table).reshape(n, width)
    cu, total, slots, taken = kda.plan_requests(ints(past), ints(new), t, ints(free), page, tokens)
    torch.cuda.synchronize()
    want = ref.plan(past, new, table, free, page, tokens)
    assert cu.tolist() == want[0]
    assert total.tolist() == want[1]
    assert slots.tolist() == want[2]
    assert t.tolist() == want[3]
    assert taken.tolist() == [want[4]]


def made(rng, n, most_past, most_new, page, spare=5, extra=0):
    past = [rng.randint(0, most_past) for _ in range(n)]
    new = [rng.randint(0, most_new) for _ in range(n)]
    width = -(-(most_past + most_new) // page) + extra
    ids = list(range(n * width + spare))
    rng.shuffle(ids)
    table = []
    for p in past:
        held = -(-p // page)
        table.append([ids.pop() for _ in range(held)] + [-1] * (width - held))
    return past, new, table, ids


@pytest.mark.parametrize("n,past,new,page", [(1, 0, 1, 16), (1, 100, 1, 64), (3, 40, 40, 16), (255, 300, 1, 64),
                                             (256, 200, 5, 32), (257, 90, 30, 16), (1000, 50, 9, 256),
                                             (8192, 20, 3, 16), (2, 5, 9000, 128)])
def test_plan(n, past, new, page):
    rng = random.Random(n + page)
    p, m, table, free = made(rng, n, past, new, page)
    check(p, m, table, free, page, sum(m))
    check(p, m, table, free, page, sum(m) + 77)         # rows behind the last request's


def test_plan_edges():
    check([], [], [], [1, 2], 16, 0)
    check([], [], [], [], 16, 5)
    check([7], [0], [[3]], [4], 16, 0)
    check([0, 0, 0], [0, 0, 0], [[-1], [-1], [-1]], [5], 16, 4)
    check([16, 15, 17], [1, 1, 1], [[9, -1], [8, -1], [7, 6]], [1, 2, 3], 16, 3)
    check([5, 6], [3, 3], [[], []], [1], 16, 6)          # no room for a page


def test_plan_bad_lengths_and_lists():
    rng = random.Random(7)
    p, m, table, free = made(rng, 40, 100, 60, 16)
    check(p, m, table, free[:30], 16, sum(m))            # the list ends
    check(p, m, table, [], 16, sum(m))
    check(p, m, table, free, 16, sum(m) // 2)            # more tokens than rows
    check([-5] + p[1:], m[:-1] + [-9], table, free, 16, sum(m))
    check([x * 3 for x in p], m, [r[:4] for r in table], free, 16, sum(m))   # longer than the table's rows
    check([2 ** 31 - 1, 2 ** 31 - 1], [2 ** 31 - 1, 5], [[1], [2]], [7, 8], 16, 30)
    check(p, m, [[-3 if i % 2 else x for i, x in enumerate(r)] for r in table], free, 16, sum(m))


def test_plan_gives_what_the_packed_calls_take():
    """The offsets feed kda_varlen_prefill as they are."""
    past, new = [0, 70, 3], [65, 1, 130]
    T, H, d = sum(new), 2, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    q, k, v, g = (r(1, T, H, d).bfloat16() for _ in range(4))
    la, beta = -torch.rand(1, T, H, d, generator=gen, device="cuda"), torch.rand(1, T, H, generator=gen, device="cuda")
    cu, _, _, _ = kda.plan_requests(ints(past), ints(new), ints([[-1] * 9, [0, 1] + [-1] * 7, [2] + [-1] * 8]),
                                    ints(list(range(3, 30))), 64, T)
    out, state = kda.varlen_prefill(q, k, v, la, beta, g, -0.1, cu)
    want, wstate = kda.varlen_prefill(q, k, v, la, beta, g, -0.1, ints([0, 65, 66, 196]))
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(state, wstate)
