"""simsd_page_map against a plain loop over the sequences (whole numbers:
equal)."""
import random

import pytest
import torch

import speculative_decoding_diffusion_gb300 as pkg

pytestmark = pytest.mark.gpu
PAGE = 16


def plain(lens, new, held, queue, ring, table, total_n, width, cap):
    """(held, queue, ring, table, served, slots) after the call, as lists."""
    head, count = queue
    ring, table, held = list(ring), [list(r) for r in table], list(held)
    slots, served = [-7] * total_n, []
    avail, take, put, c0 = count, head, head + count, 0
    short = False
    given = 0
    for b, (L, n) in enumerate(zip(lens, new)):
        need = (L + n + PAGE - 1) // PAGE
        grow = need - held[b]
        fine = True
        if grow > 0:
            if short or grow > avail:
                short, fine = True, False
            else:
                for j in range(held[b], need):
                    table[b][j] = ring[take % cap]
                    take += 1
                avail -= grow
        else:
            for j in range(need, held[b]):
                ring[put % cap] = table[b][j]
                put += 1
                given += 1
        if fine:
            held[b] = need
        for i in range(n):
            p = L + i
            slots[c0 + i] = table[b][p // PAGE] * PAGE + p % PAGE if fine else -1
        served.append(int(fine))
        c0 += n
    return held, [take % cap, avail + given], ring, table, served, slots


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class State:
    def __init__(self, rng, batch, width, spare, full):
        self.batch, self.width = batch, width
        self.held = [rng.randint(0, width if full else max(0, width // 2)) for _ in range(batch)]
        self.cap = sum(self.held) + spare
        ids = list(range(self.cap))
        rng.shuffle(ids)
        self.table = []
        for h in self.held:
            self.table.append([ids.pop() for _ in range(h)] + [0] * (width - h))
        head = rng.randrange(self.cap)
        self.ring = [-1] * self.cap
        for i, p in enumerate(ids):
            self.ring[(head + i) % self.cap] = p
        self.queue = [head, len(ids)]


def call(st, lens, new, alias, ws=None):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    total = cu[-1]
    held, queue, ring, table = i32(st.held), i32(st.queue), i32(st.ring), i32(st.table)
    held_out = held if alias else torch.full_like(held, -9)
    queue_out = queue if alias else torch.full_like(queue, -9)
    served = torch.full_like(held, -9)
    slots = torch.full((total + 3,), -7, dtype=torch.int64, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda") if ws is None else ws
    pkg.page_map(i32(lens), i32(cu), held, queue, ring, table, held_out, queue_out, served, slots, ws, total)
    return [t.tolist() for t in (held_out, queue_out, ring, table, served)] + [slots.tolist()], ws


@pytest.mark.parametrize("batch,width,spare", [(1, 1, 1), (1, 40, 50), (7, 9, 100), (300, 5, 2000), (1025, 3, 4000),
                                               (33, 300, 12000), (2500, 2, 100)])
@pytest.mark.parametrize("alias", [False, True])
def test_matches_plain_loop(batch, width, spare, alias):
    rng = random.Random(batch * 7 + spare)
    st = State(rng, batch, width, spare, full=False)
    for _ in range(3):                       # the state goes on from call to call
        lens = [rng.choice([0, rng.randint(0, width * PAGE)]) for _ in range(batch)]
        new = [rng.randint(0, min(40, width * PAGE - L)) for L in lens]
        want = plain(lens, new, st.held, st.queue, st.ring, st.table, sum(new), width, st.cap)
        got, ws = call(st, lens, new, alias)
        for g, w in zip(got[:5], want[:5]):
            assert g == w
        assert got[5][:sum(new)] == want[5] and got[5][sum(new):] == [-7, -7, -7]
        assert pkg.read_status(ws) == 0
        st.held, st.queue, st.ring, st.table = want[:4]


def test_no_pages_left_and_exactly_enough():
    st = State(random.Random(1), 4, 8, 3, full=False)
    st.held, st.table = [0, 0, 0, 0], [[0] * 8 for _ in range(4)]
    st.cap, st.ring, st.queue = 3, [2, 0, 1], [1, 3]
    lens, new = [16, 16, 17, 0], [0, 1, 0, 1]          # 1, 2, 2 and 1 pages: the third is short
    want = plain(lens, new, st.held, st.queue, st.ring, st.table, 2, 8, 3)
    got, ws = call(st, lens, new, False)
    assert got[4] == [1, 1, 0, 0] == want[4]
    assert got[:2] == [[1, 2, 0, 0], [1, 0]] and got[5][:2] == want[5] and want[5][1] == -1
    assert pkg.read_status(ws) == 0


def test_bad_numbers_are_refused_one_by_one():
    st = State(random.Random(2), 3, 4, 9, full=False)
    st.held = [0, 0, 0]
    st.cap, st.ring, st.queue = 9, list(range(9)), [0, 9]
    got, ws = call(st, [-1, 16, 65], [2, 1, 0], False)     # a negative length; more pages than the row
    assert got[4] == [0, 1, 0] and got[0] == [0, 2, 0] and got[1] == [2, 7]
    assert got[5][:3] == [-1, -1, 1 * 16]
    assert pkg.read_status(ws) == 2
    # a ring that cannot be: nothing is served
    for queue in ([9, 1], [0, 10], [-1, 2], [0, -1]):
        st.queue = queue
        got, ws = call(st, [16, 16, 16], [1, 1, 1], False)
        assert got[4] == [0, 0, 0] and got[0] == [0, 0, 0] and got[1] == queue
        assert got[2] == list(range(9)) and got[5][:3] == [-1, -1, -1]
        assert pkg.read_status(ws) == 2


def test_without_new_tokens():
    st = State(random.Random(3), 5, 6, 30, full=True)
    lens = [0, 96, 1, 17, 50]
    want = plain(lens, [0] * 5, st.held, st.queue, st.ring, st.table, 0, 6, st.cap)
    held, queue, ring, table = i32(st.held), i32(st.queue), i32(st.ring), i32(st.table)
    served = torch.empty_like(held)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    pkg.page_map(i32(lens), None, held, queue, ring, table, held, queue, served, None, ws, 0)
    assert [t.tolist() for t in (held, queue, ring, table, served)] == list(want[:5])


def test_largest_batch_and_graph_replay():
    batch, width = 16384, 2
    rng = random.Random(5)
    st = State(rng, batch, width, 40000, full=False)
    lens = [rng.randint(0, 20) for _ in range(batch)]
    new = [rng.randint(0, 12) for _ in range(batch)]
    want = plain(lens, new, st.held, st.queue, st.ring, st.table, sum(new), width, st.cap)
    got, ws = call(st, lens, new, False)
    for g, w in zip(got[:5], want[:5]):
        assert g == w
    assert got[5][:sum(new)] == want[5]
    # captured: two replays carry the aliased state on
    st = State(rng, 64, 6, 500, full=False)
    lens_t, cu_t = i32([10] * 64), i32(list(range(0, 65 * 5, 5)))
    held, queue, ring, table = i32(st.held), i32(st.queue), i32(st.ring), i32(st.table)
    served, slots = torch.empty_like(held), torch.empty(320, dtype=torch.int64, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.page_map(lens_t, cu_t, held, queue, ring, table, held, queue, served, slots, ws, 320)
    for L in (10, 33, 0):
        lens_t.fill_(L)
        want = plain([L] * 64, [5] * 64, st.held, st.queue, st.ring, st.table, 320, 6, st.cap)
        graph.replay()
        assert [t.tolist() for t in (held, queue, ring, table, served, slots)] == list(want)
        st.held, st.queue, st.ring, st.table = want[:4]


@pytest.mark.parametrize("n", [9, 10])
def test_positions_at_the_end_of_32_bits(n):
    """A row of 2^27 + 1 pages: positions up to 2^31 - 1 have a slot, a sequence that would pass it is refused."""
    width = 2 ** 27 + 1
    table = torch.zeros(1, width, dtype=torch.int32, device="cuda")
    table[0, 2 ** 27 - 1] = 5
    ring = torch.zeros(width, dtype=torch.int32, device="cuda")
    held, queue, served = i32([2 ** 27]), i32([0, 0]), i32([7])
    slots = torch.full((n,), -7, dtype=torch.int64, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    pkg.page_map(i32([2 ** 31 - 10]), i32([0, n]), held, queue, ring, table, held, queue, served, slots, ws, n)
    ok = n == 9
    assert pkg.read_status(ws) == (0 if ok else 2)
    assert served.item() == int(ok) and held.item() == 2 ** 27 and queue.tolist() == [0, 0]
    assert slots.tolist() == ([5 * PAGE + 6 + i for i in range(9)] if ok else [-1] * 10)
