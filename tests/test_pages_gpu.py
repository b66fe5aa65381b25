"""The page pool on the GPU against a plain model of it (whole numbers, equal
to the last one), and its faults."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

from mla_attention_prolog_gb300 import binding  # noqa: E402

DEV = "cuda"
SEQ, PAGE, FULL, SLOT = (binding.STATUS_SEQ_RANGE, binding.STATUS_PAGE_RANGE, binding.STATUS_POOL_FULL,
                         binding.STATUS_SLOT_RANGE)


def i32(*a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


class Model:
    """The pool's definition, one entry at a time."""

    def __init__(self, S, width, pages, page):
        self.S, self.width, self.page = S, width, page
        self.table, self.lens, self.refs = [[-1] * width for _ in range(S)], [0] * S, [0] * pages
        self.status = 0

    def held(self, n):
        return -(-n // self.page)

    def free(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def extend(self, seqs, counts, total):
        slots, pos, free, taken, seen = [-1] * total, [0] * total, self.free(), 0, set()
        lens, at = list(self.lens), 0
        for s, c in zip(seqs, counts):
            here, at = at, at + max(c, 0)
            if not 0 <= s < self.S or c < 0 or s in seen:
                self.status |= SEQ
                seen.add(s)
                continue
            seen.add(s)
            n = lens[s]
            if n + c > self.width * self.page:
                self.status |= FULL
                continue
            need = self.held(n + c) - self.held(n)
            taken += need
            if need and taken > len(free):
                self.status |= FULL
                continue
            for k in range(need):
                self.table[s][self.held(n) + k] = free[taken - need + k]
                self.refs[free[taken - need + k]] = 1
            self.lens[s] = n + c
            for j in range(n, n + c):
                if here + j - n < total:
                    slots[here + j - n] = self.table[s][j // self.page] * self.page + j % self.page
                    pos[here + j - n] = j
        if at > total:
            self.status |= SLOT
        return slots, pos

    def fork(self, parents, children):
        free, taken, seen, pairs = self.free(), 0, set(), []
        lens, table = list(self.lens), [list(r) for r in self.table]
        for a, c in zip(parents, children):
            pairs.append((-1, -1))
            ok = 0 <= a < self.S and 0 <= c < self.S and lens[c] == 0 and c not in seen
            seen.add(c)
            if not ok:
                self.status |= SEQ
                continue
            full = lens[a] // self.page
            if lens[a] % self.page:
                taken += 1
                if taken > len(free):
                    self.status |= FULL
                    continue
                self.table[c][full] = free[taken - 1]
                self.refs[free[taken - 1]] = 1
                pairs[-1] = (table[a][full], free[taken - 1])
            for j in range(full):
                self.table[c][j] = table[a][j]
                self.refs[table[a][j]] += 1
            self.lens[c] = lens[a]
        return pairs

    def release(self, seqs):
        for s in seqs:
            if not 0 <= s < self.S:
                self.status |= SEQ
                continue
            for j in range(self.held(self.lens[s])):
                self.refs[self.table[s][j]] -= 1
            self.table[s], self.lens[s] = [-1] * self.width, 0

    def compact(self):
        live = [p for p, r in enumerate(self.refs) if r]
        L = len(live)
        holes, moved = [p for p in range(L) if self.refs[p] == 0], [-1] * len(self.refs)
        k = 0
        for p in live:
            moved[p] = p
            if p >= L:
                moved[p], k = holes[k], k + 1
        refs = [0] * len(self.refs)
        for p in live:
            refs[moved[p]] = self.refs[p]
        self.refs = refs
        self.table = [[moved[p] if p >= 0 else p for p in row] for row in self.table]
        return moved, L


class Pair:
    """A pool on the GPU beside its model; every call is compared whole."""

    def __init__(self, S, width, pages, page):
        self.m = Model(S, width, pages, page)
        self.table, self.lens, self.refs = (torch.tensor(x, dtype=torch.int32, device=DEV).reshape(shape) for x, shape in (
            (self.m.table, (S, width)), (self.m.lens, (S,)), (self.m.refs, (pages,))))
        self.status = i32(0)
        self.pool = binding.PagePool(self.table, self.lens, self.refs, page, self.status)

    def same(self):
        assert self.lens.tolist() == self.m.lens
        assert self.table.tolist() == self.m.table
        assert self.refs.tolist() == self.m.refs
        assert int(self.status.item()) == self.m.status

    def extend(self, seqs, counts, total=None):
        total = sum(max(c, 0) for c in counts) if total is None else total
        slots, pos = (torch.full((total,), 77, dtype=torch.int32, device=DEV) for _ in "ab")
        self.pool.extend(i32(*seqs), i32(*counts), slots, pos)
        want = self.m.extend(seqs, counts, total)
        assert (slots.tolist(), pos.tolist()) == want
        self.same()
        return slots

    def fork(self, parents, children):
        src, dst = i32(*[9] * len(parents)), i32(*[9] * len(parents))
        self.pool.fork(i32(*parents), i32(*children), src, dst)
        assert list(zip(src.tolist(), dst.tolist())) == self.m.fork(parents, children)
        self.same()
        return src, dst

    def release(self, seqs):
        self.pool.release(i32(*seqs))
        self.m.release(seqs)
        self.same()

    def compact(self):
        moved, live = torch.full((len(self.m.refs),), 77, dtype=torch.int32, device=DEV), i32(-1)
        self.pool.compact(moved, live)
        want, L = self.m.compact()
        assert moved.tolist() == want and int(live.item()) == L
        self.same()
        return moved


@pytest.mark.parametrize("seed,S,width,pages,page", [(1, 6, 5, 20, 16), (2, 40, 12, 300, 1), (3, 300, 9, 1500, 7),
                                                     (4, 20, 40, 70000, 64), (5, 64, 20, 32768, 16)])
def test_random_steps(seed, S, width, pages, page):
    r = random.Random(seed)
    x = Pair(S, width, pages, page)
    for _ in range(25):
        op = r.choice(["extend", "extend", "fork", "release", "compact"])
        if op == "extend":
            seqs = r.sample(range(S), r.randint(1, min(S, 60)))
            x.extend(seqs, [r.choice([0, 1, r.randint(0, 2 * page + 1), r.randint(0, width * page)]) for _ in seqs])
        elif op == "fork":
            empty = [s for s in range(S) if x.m.lens[s] == 0]
            children = r.sample(empty, r.randint(0, min(len(empty), 10)))
            x.fork([r.randrange(S) for _ in children], children)
        elif op == "release":
            x.release(r.sample(range(S), r.randint(0, S // 2)))
        else:
            x.compact()


def test_first_pages_of_a_high_pool():
    """Live pages in several passes of the scan move down across them."""
    pages = 100_000
    x = Pair(3, 60_000, pages, 1)
    x.extend([0, 1, 2], [40_000, 20_000, 39_000])
    x.release([0])
    x.compact()
    x.extend([0], [41_000], total=41_500)
    x.release([1])
    x.compact()


def test_extend_refusals_leave_the_rest():
    x = Pair(6, 4, 9, 16)
    x.extend([0, 1, 0, 7, -1, 2], [16, 17, 5, 1, 1, 0])   # 0 twice, 7 and -1 outside
    assert x.m.status == SEQ
    x.extend([3, 4, 5], [65, 64, 48])                     # 65 > 4 pages; 64 takes 4; 48 needs 3 of the 2 left
    assert x.m.status == SEQ | FULL
    x.extend([5, 1], [-3, 2], total=10)
    x.extend([2], [20], total=3)                          # more tokens than slots asked for
    assert x.m.status & SLOT


def test_extend_without_buffers():
    """Growing sequences needs neither slots nor positions."""
    x = Pair(3, 4, 9, 16)
    x.pool.extend(i32(0, 2), i32(20, 3))
    x.m.extend([0, 2], [20, 3], 23)
    x.same()
    positions = i32(*[9] * 7)
    x.pool.extend(i32(2), i32(7), positions=positions)
    assert positions.tolist() == x.m.extend([2], [7], 7)[1]
    x.same()


def test_lists_of_any_length():
    """As many entries as a call takes, and repeats far apart."""
    r = random.Random(9)
    x = Pair(1200, 3, 2500, 16)
    seqs = r.sample(range(1200), 1023)
    x.extend(seqs + [seqs[5]], [r.randint(0, 20) for _ in range(1024)])
    empty = [s for s in range(1200) if x.m.lens[s] == 0]
    x.fork([r.randrange(1200) for _ in empty], empty)
    x.release(seqs[:600] + seqs[:424])
    x.compact()


def test_fork_refusals_leave_the_rest():
    x = Pair(8, 4, 10, 16)
    x.extend([0, 1], [40, 32])
    x.fork([0, 1, 0, 9, 0, 2, 0], [2, 3, 2, 4, 0, 5, -1])  # 2 twice, parent 9, child 0 in use, an empty parent, child -1
    assert x.m.status == SEQ
    x.fork([0, 0, 0, 0, 0], [4, 5, 6, 7, 5])               # 3 + 2 + 1 pages in use, 4 more: the pool is just full
    assert x.m.status == SEQ and not x.m.free()
    x = Pair(8, 4, 9, 16)
    x.extend([0, 1], [40, 32])
    x.fork([0, 1, 0, 0, 0, 0, 1], [2, 3, 4, 5, 6, 7, 7])   # 4 free pages: child 7 gets none; 7 again is refused
    assert x.m.status == SEQ | FULL


def test_release_twice_and_outside():
    x = Pair(5, 4, 20, 16)
    x.extend([0, 1], [40, 33])
    x.fork([0], [2])
    x.release([0, 0, 4, 17, -1, 0])
    assert x.m.status == SEQ
    x.compact()


def test_empty_calls():
    x = Pair(2, 2, 4, 16)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    x.pool.release(none)
    x.pool.fork(none, none, none, none)
    x.pool.extend(none, none)
    x.same()
    x.compact()
    slots = x.extend([], [], total=5)
    assert slots.tolist() == [-1] * 5


@pytest.mark.parametrize("layers", [None, 1, 3])
@pytest.mark.parametrize("page,width", [(16, 576), (64, 576), (3, 8), (1, 8)])
def test_copy_pages(layers, page, width):
    g = torch.Generator(DEV).manual_seed(1)
    shape = ([] if layers is None else [layers]) + [50, page, width]
    cache = torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)
    want = cache.clone()
    src, dst = [3, 7, -1, 9, 4, 3, 11], [20, 21, 22, -1, 4, 23, 0]
    c, w = (t if layers is None else t.transpose(0, 1) for t in (cache.clone(), want))
    for a, b in zip(src, dst):
        if a >= 0 and b >= 0:
            w[b] = c[a]
    status = i32(0)
    binding.copy_pages(cache, i32(*src), i32(*dst), status=status)
    assert torch.equal(cache.view(torch.int16), want.view(torch.int16)) and int(status.item()) == 0
    binding.copy_pages(cache, i32(50, 1), i32(2, 1000), status=status)
    assert torch.equal(cache.view(torch.int16), want.view(torch.int16)) and int(status.item()) == PAGE
    moved = torch.arange(50, dtype=torch.int32, device=DEV)
    moved[49], moved[48] = 1, -1
    (want if layers is None else want.transpose(0, 1))[1] = (want if layers is None else want.transpose(0, 1))[49].clone()
    binding.copy_pages(cache, None, moved)
    assert torch.equal(cache.view(torch.int16), want.view(torch.int16))


def test_copy_pages_behind_32_bit_offsets():
    pages = (1 << 32) // (64 * 576 * 2) + 50
    cache = torch.zeros((2, pages, 64, 576), dtype=torch.bfloat16, device=DEV)
    cache[1, pages - 1] = 3.0
    cache[0, 2] = 5.0
    binding.copy_pages(cache, i32(pages - 1, 2), i32(pages - 3, pages - 2))
    assert (cache[1, pages - 3] == 3).all() and (cache[0, pages - 2] == 5).all() and (cache[0, pages - 3] == 0).all()


def test_bad_pages_in_a_table():
    """A corrupt table entry is counted nowhere and sets the status."""
    x = Pair(3, 4, 8, 16)
    x.extend([0], [40])
    x.table[0, 1] = 99
    x.pool.release(i32(0))
    assert int(x.status.item()) == PAGE and x.refs.tolist() == [0, 1, 0, 0, 0, 0, 0, 0]
    y = Pair(3, 4, 8, 16)
    y.extend([0], [40])
    y.table[0, 0] = 8
    moved = i32(*[0] * 8)
    y.pool.compact(moved)
    assert int(y.status.item()) == PAGE


def test_a_captured_step():
    """fork, extend and compact in one graph: the replay follows the state."""
    x = Pair(8, 6, 64, 16)
    x.extend([0, 1], [40, 20])
    a, b, src, dst = i32(0), i32(3), i32(0), i32(0)
    seqs, counts, slots, moved = i32(0, 3), i32(9, 9), i32(*[0] * 18), i32(*[0] * 64)
    state = [t.clone() for t in (x.table, x.lens, x.refs)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.pool.fork(a, b, src, dst)
        x.pool.extend(seqs, counts, slots)
        x.pool.compact(moved)
    for t, u in zip((x.table, x.lens, x.refs), state):
        assert torch.equal(t, u)   # captured, not run
    for child in (3, 4):
        b.fill_(child)
        seqs.copy_(i32(0, child))
        g.replay()
        torch.cuda.synchronize()
        pairs = x.m.fork([0], [child])
        want, _ = x.m.extend([0, child], [9, 9], 18)
        assert [(int(src.item()), int(dst.item()))] == pairs and slots.tolist() == want
        assert moved.tolist() == x.m.compact()[0]
        x.same()


def test_steps_that_follow_one_another():
    """Launches overlap the end of the ones before them: steps of all calls in a
    row leave what they leave with a synchronize between any two."""
    ends = []
    for apart in (False, True):
        S, width, pages, page = 12, 8, 90, 16
        table = torch.full((S, width), -1, dtype=torch.int32, device=DEV)
        lens, refs = i32(*[0] * S), i32(*[0] * pages)
        pool = binding.PagePool(table, lens, refs, page)
        g = torch.Generator(DEV).manual_seed(5)
        cache = torch.randint(-2 ** 15, 2 ** 15, (2, pages, page, 8), generator=g, device=DEV).to(torch.int16).view(torch.bfloat16)
        src, dst, moved, slots, pos = i32(-1, -1), i32(-1, -1), i32(*[0] * pages), i32(*[0] * 40), i32(*[0] * 40)
        args = [(i32(k % 4, 4 + k % 4), i32(7, 11), i32(k % 4, 4 + k % 4), i32(8 + k % 4, 8 + (k + 1) % 4)) for k in range(30)]
        torch.cuda.synchronize()
        for seqs, counts, parents, children in args:
            for call in (lambda: pool.extend(seqs, counts, slots, pos), lambda: pool.release(children),
                         lambda: pool.fork(parents, children, src, dst), lambda: binding.copy_pages(cache, src, dst),
                         lambda: pool.compact(moved), lambda: binding.copy_pages(cache, None, moved)):
                call()
                if apart:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        ends.append([t.clone() for t in (table, lens, refs, cache.view(torch.int16), slots, pos, moved, src, dst)])
    assert all(torch.equal(a, b) for a, b in zip(*ends)) and ends[0][1].sum() > 0
