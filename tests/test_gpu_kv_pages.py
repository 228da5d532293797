"""fh_kv_pages_update against the documented rules, one page after another."""
import numpy as np
import pytest
import torch

from _gpu_util import fh
from _kv_ref import pages_update

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device="cuda")


def start(rng, n, page, held, spare, width_extra=2, target=None):
    """A consistent state: every request holds the pages of its tokens, the others are free."""
    held = np.asarray(held)
    hp = -(-np.maximum(held, 0) // page)
    width = int(max(hp.max(initial=0), (-(-np.maximum(target, 0) // page)).max(initial=0))) + width_extra
    total = int(hp.sum()) + spare
    order = rng.permutation(total)
    table = np.full((n, width), -7, np.int64)
    at = 0
    for b in range(n):
        table[b, :hp[b]] = order[at:at + hp[b]]
        at += hp[b]
    free = np.full(max(total, 1), -9, np.int64)
    free[:total - at] = order[at:]
    return table, free, total - at


def run(held, target, table, free, count, page, cap, alias=False):
    m = fh()
    n = len(held)
    d = dict(held=i32(held), target=i32(target), table=i32(table), free=i32(free), count=i32([count]))
    lens = d["held"] if alias else i32(np.full(n, 77))
    out = d["count"] if alias else i32([-5])
    q_starts, status = i32(np.full(n + 1, 77)), i32([99])
    slots = torch.full((cap + 8,), 12345, dtype=torch.int64, device="cuda")
    m.fh_kv_pages_update(d["held"], d["target"], d["table"], d["free"], d["count"], out, lens, q_starts, slots[:cap],
                         status, page)
    torch.cuda.synchronize()
    assert (slots[cap:] == 12345).all()
    return (int(status), d["table"].cpu().numpy(), d["free"].cpu().numpy(), int(out), lens.cpu().numpy(),
            q_starts.cpu().numpy(), slots[:cap].cpu().numpy())


def check(held, target, table, free, count, page, cap, alias=False):
    ref = pages_update(held, target, table, free, count, page, cap, table.shape[1])
    got = run(held, target, table, free, count, page, cap, alias)
    for name, r, g in zip(("status", "table", "free", "count", "lens", "q_starts", "slots"), ref, got):
        np.testing.assert_array_equal(g, r, err_msg=name)
    return got


def mixed(rng, n, page, most, grow):
    held = rng.integers(0, most + 1, n)
    target = held + rng.integers(0, grow + 1, n)
    kind = rng.integers(0, 6, n)
    target = np.where(kind == 0, 0, target)
    target = np.where(kind == 1, rng.integers(0, held + 1), target)
    return held, target


@pytest.mark.parametrize("n,page,most,grow", [(1, 16, 0, 1), (1, 16, 40, 1), (1, 1, 5, 3), (3, 16, 100, 33),
                                              (33, 32, 500, 1), (256, 16, 700, 5), (1000, 64, 900, 130),
                                              (1025, 16, 60, 40), (8192, 16, 40, 20), (7, 1024, 5000, 3000)])
@pytest.mark.parametrize("alias", [False, True])
def test_mixed_steps(n, page, most, grow, alias):
    rng = np.random.default_rng(n * 7 + page)
    held, target = mixed(rng, n, page, most, grow)
    need = int(np.maximum(-(-target // page) - -(-held // page), 0).sum())
    table, free, count = start(rng, n, page, held, need + 3, target=target)
    rows = int(np.maximum(target - held, 0).sum())
    check(held, target, table, free, count, page, rows + 5, alias)


def test_growth_served_by_pages_given_back_in_the_same_step():
    rng = np.random.default_rng(1)
    held, target = np.array([100, 5, 64, 0]), np.array([0, 90, 16, 33])
    table, free, count = start(rng, 4, 16, held, 2, target=target)
    status, *_ = check(held, target, table, free, count, 16, 200)
    assert status == 0


def test_pool_used_up_exactly_and_one_page_short():
    rng = np.random.default_rng(2)
    held, target = np.array([16, 20]), np.array([17, 49])
    table, free, count = start(rng, 2, 16, held, 3, target=target)
    assert check(held, target, table, free, count, 16, 64)[0] == 0
    table, free, count = start(rng, 2, 16, held, 2, target=target)
    assert check(held, target, table, free, count, 16, 64)[0] == fh().FH_KV_NO_PAGES


@pytest.mark.parametrize("alias", [False, True])
def test_refused_steps_leave_everything_as_it_was(alias):
    m = fh()
    rng = np.random.default_rng(3)
    held, target = np.array([30, 5, 50]), np.array([60, 6, 0])
    table, free, count = start(rng, 3, 16, held, 8, target=target)
    assert check(held, target, table, free, count, 16, 30, alias)[0] == m.FH_KV_SLOTS_FULL   # 31 new tokens
    assert check(held, target, table, free, count, 16, 31, alias)[0] == 0
    assert check(held, np.array([60, -1, 0]), table, free, count, 16, 64, alias)[0] == m.FH_KV_BAD_LENGTH
    assert check(np.array([30, -5, 50]), target, table, free, count, 16, 64, alias)[0] == m.FH_KV_BAD_LENGTH
    assert check(held, np.array([10 ** 9, 6, 0]), table, free, count, 16, 64, alias)[0] & m.FH_KV_TABLE_FULL
    assert check(held, target, table, free, len(free), 16, 64, alias)[0] == m.FH_KV_STACK_OVERFLOW
    assert check(held, target, table, free, -1, 16, 64, alias)[0] & m.FH_KV_STACK_OVERFLOW
    big = np.array([2 ** 31 - 1] * 3)
    assert check(held, big, table, free, count, 16, 64, alias)[0] & m.FH_KV_TABLE_FULL


@pytest.mark.parametrize("cap", [8192, 8193, 40000])
def test_slots_of_one_launch_and_of_two(cap):
    """Capacities at the border of the one-launch form; served, refused, and with no new token at all."""
    rng = np.random.default_rng(cap)
    held, target = mixed(rng, 300, 16, 400, 40)
    need = int(np.maximum(-(-target // 16) - -(-held // 16), 0).sum())
    table, free, count = start(rng, 300, 16, held, need, target=target)
    assert check(held, target, table, free, count, 16, cap, True)[0] == 0
    assert check(held, held + 17, table, free, 5, 16, cap, True)[0] == fh().FH_KV_NO_PAGES  # 300 pages and more, of 5
    assert check(held, held, table, free, count, 16, cap, True)[0] == 0
    held, target = np.array([10, 3, 7]), np.array([10 + cap - 5, 0, 7 + 5])  # the capacity to the last slot
    table, free, count = start(rng, 3, 16, held, cap // 16 + 3, target=target)
    assert check(held, target, table, free, count, 16, cap)[0] == 0


def test_no_new_tokens_and_no_slots():
    rng = np.random.default_rng(4)
    held = np.array([3, 40, 0])
    table, free, count = start(rng, 3, 16, held, 1, target=held)
    check(held, held, table, free, count, 16, 0)
    check(held, held, table, free, count, 16, 300)


def test_same_inputs_again_give_the_same():
    m = fh()
    rng = np.random.default_rng(5)
    held, target = mixed(rng, 200, 16, 300, 40)
    table, free, count = start(rng, 200, 16, held, 4000, target=target)
    d = [i32(x) for x in (held, target, table, free, [count])]
    out, lens, qs, status = i32([0]), i32(np.zeros(200)), i32(np.zeros(201)), i32([0])
    slots = torch.zeros(9000, dtype=torch.int64, device="cuda")
    seen = []
    for _ in range(3):
        m.fh_kv_pages_update(*d, out, lens, qs, slots, status, 16)
        seen.append([x.clone() for x in (d[2], d[3], out, lens, qs, slots, status)])
    for a in seen[1:]:
        assert all(torch.equal(x, y) for x, y in zip(seen[0], a))


def test_unknown_page_gives_no_slot():
    """A table entry below 0 where held tokens end inside a page: their new neighbours get no slot."""
    table = np.full((1, 4), -1)
    got = run([5], [20], table, np.array([3, 2, 1]), 3, 16, 20)
    assert got[0] == 0 and (got[6][:11] == -1).all() and got[6][11:15].tolist() == [16, 17, 18, 19]


def test_captured_steps_with_many_slots():
    """The two-launch form captured in a graph, counts and lengths updated in place from replay to replay."""
    m = fh()
    rng = np.random.default_rng(6)
    n, page, cap = 500, 16, 30000
    state = [np.zeros(n, np.int64), np.full((n, 40), -1, np.int64), rng.permutation(9000), 9000]
    target, held, table, free, count = i32(state[0]), i32(state[0]), i32(state[1]), i32(state[2]), i32([9000])
    qs, status, slots = i32(np.zeros(n + 1)), i32([0]), torch.zeros(cap, dtype=torch.int64, device="cuda")
    call = lambda: m.fh_kv_pages_update(held, target, table, free, count, count, held, qs, slots, status, page)
    call()  # nothing moves
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(6):
        want = np.maximum(0, state[0] + rng.integers(-60, 110, n)).clip(max=600)
        target.copy_(i32(want))
        graph.replay()
        torch.cuda.synchronize()
        ref = pages_update(state[0], want, state[1], state[2], state[3], page, cap, 40)
        assert ref[0] == 0 and int(status) == 0
        for r, g in zip(ref[1:], (table, free, count, held, qs, slots)):
            np.testing.assert_array_equal(g.cpu().numpy().reshape(np.shape(r)), r)
        state = [ref[4], ref[1], ref[2], ref[3]]


def test_as_many_pages_as_the_sizes_allow():
    """2^31 - 1 pages of one token taken in one step and given back in the next: the last threads' next entry would be
    past 32 bits."""
    m = fh()
    n, half = 2 ** 31 - 1, 2 ** 30
    held, target = i32([0, 0]), i32([half, half - 1])
    table = torch.full((2, half), -7, dtype=torch.int32, device="cuda")
    free = torch.arange(n, dtype=torch.int32, device="cuda")
    count, starts, status = i32([n]), i32([0, 0, 0]), i32([9])
    slots = torch.zeros(n, dtype=torch.int64, device="cuda")

    def down(t):
        """t[i] == n - 1 - i throughout."""
        step = 1 << 28
        return all(torch.equal(t[a:a + step], torch.arange(n - 1 - a, n - 1 - min(a + step, n), -1, dtype=t.dtype,
                                                           device="cuda")) for a in range(0, n, step))

    def step():
        m.fh_kv_pages_update(held, target, table, free, count, count, held, starts, slots, status, 1)
        return int(status), int(count), held.tolist(), starts.tolist()
    assert step() == (0, 0, [half, half - 1], [0, half, n])
    assert down(table.view(-1)[:n]) and int(table[1, -1]) == -7 and down(slots)
    assert int(free[0]) == 0 and int(free[-1]) == n - 1
    target.zero_()
    assert step() == (0, n, [0, 0], [0, 0, 0])
    assert down(free) and down(table.view(-1)[:n])
    assert int(slots.max()) == -1 and int(slots.min()) == -1
