"""Block tables and slot maps against the plain forms, one request after the other."""
import random

import pytest
import torch

import _tables as plain
import exact_attention_online_gb300 as fa

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class State:
    def __init__(self, lens, ps, max_pages, spare, seed):
        r = random.Random(seed)
        have = [plain.up(n, ps) for n in lens]
        self.ps, self.mp, self.P = ps, max_pages, max(1, sum(have) + spare)
        order = list(range(sum(have) + spare))       # (a pool without pages is refused)
        r.shuffle(order)
        self.table = [[order.pop() for _ in range(h)] + [-1] * (max_pages - h) for h in have]
        self.lens, self.n_free = list(lens), len(order)
        self.free = order + [-7] * (self.P - len(order))
        self.gpu = [i32(self.table), i32(self.lens), i32(self.free), i32([self.n_free])]

    def same(self):
        table, lens, free, n_free = (t.tolist() for t in self.gpu)
        assert lens == self.lens and n_free == [self.n_free]
        assert table == self.table and free == self.free

    def reserve(self, new, layout=None, rows=0):
        """layout: None, "padded" (rows a sequence) or "packed" (rows in all)."""
        B = len(new)
        out = [torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (B, B, B + 1)]
        kw = {}
        if layout:
            shape = (B, rows) if layout == "padded" else (rows,)
            kw = {"positions": torch.full(shape, -9, dtype=torch.int32, device="cuda"),
                  "slots": torch.full(shape, -9, dtype=torch.int64, device="cuda")}
        fa.fa_kv_reserve(*self.gpu, i32(new), *out, self.ps, **kw)
        self.n_free, starts, counts = plain.reserve(self.table, self.lens, self.free, self.n_free,
                                                    new, self.ps)
        self.same()
        cu = [0]
        for c in counts:
            cu.append(cu[-1] + c)
        assert [t.tolist() for t in out] == [starts, counts, cu]
        if layout:
            self.map_is(kw["positions"], kw["slots"], starts, counts, layout, rows)
            again = [torch.full_like(kw[k], -9) for k in ("positions", "slots")]
            if layout == "padded":
                fa.fa_kv_slots(self.gpu[0], out[0], out[1], *again, self.ps)
            else:
                fa.fa_kv_slots_varlen(self.gpu[0], out[0], out[2], *again, self.ps)
            assert torch.equal(again[0], kw["positions"]) and torch.equal(again[1], kw["slots"])
        return counts

    def map_is(self, positions, slots, starts, counts, layout, rows):
        new = plain.slots(self.table, starts, counts, self.ps)
        if layout == "padded":
            want = [(x + [(0, -1)] * rows)[:rows] for x in new]
            want = [y for x in want for y in x]
        else:
            want = [y for x in new for y in x]
            want += [(0, -1)] * (rows - len(want))
        assert positions.flatten().tolist() == [w[0] for w in want]
        assert slots.flatten().tolist() == [w[1] for w in want]

    def release(self, keep, pinned=None):
        fa.fa_kv_release(*self.gpu, i32(keep), self.ps,
                         pinned=None if pinned is None else i32(pinned))
        self.n_free = plain.release(self.table, self.lens, self.free, self.n_free, keep, self.ps,
                                    pinned)
        self.same()


@pytest.mark.parametrize("layout", ["padded", "packed"])
@pytest.mark.parametrize("B,ps,hi,new,spare", [
    (1, 16, 0, 1, 1), (1, 16, 0, 1, 0), (1, 256, 1000, 300, 5), (3, 32, 31, 1, 2),
    (64, 16, 300, 1, 64), (64, 16, 300, 4, 5), (33, 64, 500, 200, 40), (1025, 16, 40, 3, 100),
    (4096, 16, 20, 20, 2000),
])
def test_steps(B, ps, hi, new, spare, layout):
    """Several steps with requests of 0 .. new tokens, some of them refused, and rollbacks."""
    r = random.Random(B + ps + spare)
    s = State([r.randint(0, hi) for _ in range(B)], ps, plain.up(hi + 3 * new, ps), spare, 1)
    refused = 0
    for step in range(4):
        want = [r.choice([0, new, r.randint(0, new), -5]) for _ in range(B)]
        rows = new if layout == "padded" else max(1, sum(max(x, 0) for x in want)) + step
        got = s.reserve(want, layout, rows)
        refused += sum(max(x, 0) > g for x, g in zip(want, got))
        s.release([n - r.choice([0, 0, 1, new, 10 ** 6]) for n in s.lens])
    assert fa.fa_device_status() == 0
    if spare * ps < B * new // 4:
        assert refused                              # the pages did run out


def test_table_too_short():
    s = State([30, 16, 0, 32], 16, 2, 10, 3)
    assert s.reserve([3, 16, 33, 1], "padded", 16) == [0, 16, 0, 0]
    assert s.reserve([2, 1, 32, 2 ** 31 - 1], "packed", 40) == [2, 0, 32, 0]


def test_pages_run_out_in_order():
    """Sequence 1 takes the last pages, 2 gets none, 3 needs none, 4 comes too late."""
    s = State([15, 0, 0, 5, 0], 16, 8, 4, 4)
    assert s.reserve([17, 33, 16, 11, 1], "packed", 80) == [17, 33, 0, 11, 0]
    assert s.n_free == 0
    s.release([0] * 5)
    assert s.reserve([1, 1, 1, 1, 1]) == [1] * 5


def test_map_of_more_rows_than_one_launch_writes():
    for layout, rows in (("packed", 90001), ("padded", 30001)):
        s = State([5, 0, 100], 16, 4000, 5650, 5)
        assert s.reserve([30000, 1, 60000], layout, rows) == [30000, 1, 60000]


def test_padded_rows_fewer_than_the_tokens():
    s = State([5, 0], 16, 8, 9, 6)
    s.reserve([30, 2], "padded", 7)


def test_pinned_pages_stay_taken():
    s = State([100, 40, 64], 16, 8, 3, 7)
    s.release([50, 0, 0], pinned=[2, 1, 9])
    s.release([0, 0, 0], pinned=[0, 0, 0])


def test_release_of_what_is_not_there():
    s = State([0, 5, 0], 16, 4, 3, 8)
    s.release([3, 100, -4])
    s.release([-1, 0, 0])


def test_replayed_and_on_another_stream():
    """A captured step (reserve, release) replayed with other contents, and one on a side stream."""
    r = random.Random(9)
    lens = [r.randint(0, 100) for _ in range(20)]
    s = State(lens, 16, 16, 40, 9)
    new, keep = i32([0] * 20), i32([0] * 20)
    starts, counts, cu = i32([0] * 20), i32([0] * 20), i32([0] * 21)
    pos, slots = torch.zeros(300, dtype=torch.int32, device="cuda"), \
        torch.zeros(300, dtype=torch.int64, device="cuda")
    saved = [t.clone() for t in s.gpu]

    def step():
        fa.fa_kv_reserve(*s.gpu, new, starts, counts, cu, 16, positions=pos, slots=slots)
        fa.fa_kv_release(*s.gpu, keep, 16)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()                                      # with nothing to do but cut all to 0
    torch.cuda.synchronize()
    assert s.gpu[1].tolist() == [0] * 20
    for t, x in zip(s.gpu, saved):
        t.copy_(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(5):
        want = [r.randint(0, 9) for _ in range(20)]
        new.copy_(i32(want))
        s.n_free, st, c = plain.reserve(s.table, s.lens, s.free, s.n_free, want, 16)
        mine = plain.slots(s.table, st, c, 16)
        back = [n - r.randint(0, 3) for n in s.lens]
        keep.copy_(i32(back))
        s.n_free = plain.release(s.table, s.lens, s.free, s.n_free, back, 16)
        graph.replay()
        torch.cuda.synchronize()
        s.same()
        flat = [y for x in mine for y in x]
        assert slots.tolist()[:len(flat)] == [y[1] for y in flat]


def test_bad_contents_stay_inside():
    """Lengths, counts, pages and n_free outside their ranges: nothing is written outside the
    tensors (guarded rows around each)."""
    B, mp, P = 5, 4, 12
    names = {"table": B * mp, "lens": B, "free": P, "n_free": 1, "new": B, "starts": B,
             "counts": B, "cu": B + 1, "pos": 40}
    big = {}
    for n, size in names.items():
        big[n] = torch.full((size + 128,), 77, dtype=torch.int32, device="cuda")
    slots = torch.full((40 + 128,), 77, dtype=torch.int64, device="cuda")
    r = random.Random(2)
    junk = [-2 ** 31, -1, 0, 3, 17, 63, 64, 65, 10 ** 6, 2 ** 31 - 1]

    def view(n):
        return big[n][64:64 + names[n]]

    for _ in range(30):
        for n in names:
            view(n).copy_(i32([r.choice(junk) for _ in range(names[n])]))
        args = [view("table").view(B, mp), view("lens"), view("free"), view("n_free")]
        fa.fa_kv_reserve(*args, view("new"), view("starts"), view("counts"), view("cu"), 16,
                         positions=view("pos"), slots=slots[64:104])
        view("lens").copy_(i32([r.choice(junk) for _ in range(B)]))
        view("n_free").copy_(i32([r.choice(junk)]))
        fa.fa_kv_release(*args, view("new"), 16, pinned=view("starts"))
        view("cu").copy_(i32([r.choice(junk) for _ in range(B + 1)]))
        view("counts").copy_(i32([r.choice(junk) for _ in range(B)]))
        fa.fa_kv_slots_varlen(args[0], view("starts"), view("cu"), view("pos"), slots[64:104], 16)
        fa.fa_kv_slots(args[0], view("starts"), view("counts"), view("pos").view(B, 8),
                       slots[64:104].view(B, 8), 16)
        torch.cuda.synchronize()
        for n, size in names.items():
            assert (big[n][:64] == 77).all() and (big[n][64 + size:] == 77).all()
        assert (slots[:64] == 77).all() and (slots[104:] == 77).all()
