"""The page table and the store of rows on the GPU against a plain Python table (pages_ref): every
result is compared for equality."""
import random

import pytest

import pages_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def rt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from accelerator_decode_gb300 import runtime
    return runtime


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def same(t, m):
    assert t.table.cpu().tolist() == m.table()
    assert t.lens.cpu().tolist() == m.lens


def extend(t, m, slots, counts, n_rows):
    got = [x.cpu().tolist() for x in t.extend(i32(slots), i32(counts), n_rows)]
    assert got == [list(x) for x in m.extend(slots, counts, n_rows)]


def word(m):
    return sum({"position": 2, "slot": 8, "pages": 32}[w] for w in m.word)


@pytest.mark.parametrize("page,seed", [(16, 0), (16, 1), (32, 2), (128, 3), (1024, 4)])
def test_plans_of_every_kind(rt, page, seed):
    """Extends, shares and truncates in random order, with counts of zero, full pools and bad calls
    among them: tables, lengths, rows and the error word after each."""
    r = random.Random(seed)
    n_slots, max_pages = 9, 7
    n_pages = r.choice([20, 40])
    t, m = rt.PageTable(n_slots, n_pages, page, max_pages), ref.Table(n_slots, n_pages, page, max_pages)
    same(t, m)
    for step in range(120):
        n = r.randint(1, n_slots)
        slots = r.sample(range(n_slots), n)
        if r.random() < 0.1:
            slots[r.randrange(n)] = r.choice([-1, n_slots, slots[0], 1 << 30])
        what = r.random()
        if what < 0.5:
            counts = [r.choice([0, 1, r.randint(0, 2 * page), r.randint(0, 9)]) for _ in slots]
            if r.random() < 0.1:
                counts[r.randrange(n)] = r.choice([-1, -2 ** 31, max_pages * page + 1, max_pages * page, 2 ** 31 - 1])
            total = sum(c for c in counts if 0 <= c <= max_pages * page)
            extend(t, m, slots, counts, r.choice([total, total + 5, max(0, total - 3)]))
        elif what < 0.65:
            source, k = r.randrange(n_slots), r.randint(0, 3)
            t.share(i32(slots), source, k)
            m.share(slots, source, k)
        else:
            lens = [max(0, m.lens[s] - r.choice([0, 1, 5, page, 10 ** 6])) if 0 <= s < n_slots else 3 for s in slots]
            if r.random() < 0.1:
                lens[r.randrange(n)] = -7
            if r.random() < 0.2:
                lens = None
            t.truncate(i32(slots), None if lens is None else i32(lens))
            m.truncate(slots, lens)
        same(t, m)
        assert t.device_error()[1] == word(m)
        m.word.clear()


@pytest.mark.parametrize("n,rows,page", [(1024, 37, 16), (1000, 1, 16), (3, 40000, 16), (257, 700, 64)])
def test_many_sequences_and_many_rows(rt, n, rows, page):
    """Plans of several CTAs; taken back and planned again the same rows get the same pages, with a
    prefix that all share and give back together."""
    r = random.Random(n)
    most = -(-(rows + 4 * page) // page) + 1
    counts = [r.randint(max(0, rows - 50), rows) for _ in range(n - 1)]
    slots = list(range(1, n))
    r.shuffle(slots)
    total = 4 + sum(-(-c // page) for c in counts)
    t, m = rt.PageTable(n, total, page, most), ref.Table(n, total, page, most)
    m.holders = lambda p: 0 if m.given[p] == 0 else m.given[p]
    extend_fast(t, m, [0], [4 * page])
    t.share(i32(slots), 0, 4)
    for s in slots:
        m.pages[s], m.lens[s] = m.pages[0][:4], 4 * page
    for _ in range(2):
        first = extend_fast(t, m, slots, counts)
        same(t, m)
        t.truncate(i32(slots), i32([4 * page] * len(slots)))
        for s in reversed(slots):
            while len(m.pages[s]) > 4:
                m.free.append(m.pages[s].pop())
            m.lens[s] = 4 * page
        same(t, m)
    assert extend_fast(t, m, slots, counts) == first
    t.truncate(i32([0] + slots))                       # the prefix goes back once, with its first entry
    assert (t.table == -1).all() and (t.lens == 0).all()
    order = m.pages[0] + [p for s in slots for p in m.pages[s][4:]]
    m.free += order[::-1]
    m.pages, m.lens = [[] for _ in m.pages], [0] * n
    extend_fast(t, m, [1], [min(total, most) * page])
    same(t, m)
    assert t.device_error() == (0, 0)


def extend_fast(t, m, slots, counts):
    """extend() for good arguments, without the reference's search for holders."""
    got = [x.cpu().tolist() for x in t.extend(i32(slots), i32(counts), sum(counts))]
    rows, offsets = [], [0]
    for s, c in zip(slots, counts):
        for x in range(m.lens[s], m.lens[s] + c):
            if x % m.page == 0:
                m.pages[s].append(m.free.pop())
            rows.append(m.pages[s][x // m.page] * m.page + x % m.page)
        m.lens[s] += c
        offsets.append(len(rows))
    assert got == [rows, offsets, [m.lens[s] for s in slots]]
    return got


def test_a_partly_filled_shared_page_takes_no_rows(rt):
    t, m = rt.PageTable(3, 9, 16, 4), ref.Table(3, 9, 16, 4)
    extend(t, m, [0], [40], 40)
    for x in (t, m):
        x.share(i32([1]) if x is t else [1], 0, 2)
        x.truncate(i32([1]) if x is t else [1], i32([20]) if x is t else [20])
    extend(t, m, [1, 0], [1, 1], 2)                     # slot 1 would write into slot 0's second page
    assert t.device_error()[1] == 2
    same(t, m)
    for x in (t, m):
        x.truncate(i32([0]) if x is t else [0])
    extend(t, m, [1], [1], 1)                           # its own now
    same(t, m)
    assert t.device_error() == (0, 0)


def test_spoilt_tables_stay_inside(rt):
    """Entries and lengths that the caller spoilt: errors, and nothing outside the arrays is touched."""
    t = rt.PageTable(4, 8, 16, 4)
    t.extend(i32([0, 1]), i32([40, 20]), 60)
    t.table[0, 2] = 99
    t.table[1, 0] = -5
    t.truncate(i32([0, 1]))
    assert t.device_error()[1] == 2
    t.lens[2] = 1 << 20
    t.lens[3] = -4
    rows, _, lens = t.extend(i32([2, 3]), i32([1, 1]), 2)
    assert rows.tolist() == [-1, -1] and t.device_error()[1] == 2
    t.truncate(i32([2, 3]))
    assert t.device_error()[1] == 2
    t.share(i32([1]), 2, 4)
    assert t.device_error()[1] == 2


def test_captured_plans_replay(rt):
    t, m = rt.PageTable(5, 40, 16, 8), ref.Table(5, 40, 16, 8)
    slots, counts, base = i32([3, 1, 4]), i32([5, 0, 17]), i32([0, 0, 0])
    t.extend(slots, counts, 22)
    t.truncate(slots)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.truncate(slots, base)
        rows, offsets, lens = t.extend(slots, counts, 22)
    for k in range(4):
        counts.copy_(i32([5 + k, k, 17 - k]))
        base.copy_(i32([3 * k, 0, k]))
        g.replay()
        m.truncate([3, 1, 4], [3 * k, 0, k])
        want = m.extend([3, 1, 4], [5 + k, k, 17 - k], 22)
        assert [x.cpu().tolist() for x in (rows, offsets, lens)] == [list(x) for x in want]
        same(t, m)
    assert t.device_error()[1] == 0


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype,heads,page", [("bf16", 1, 16), ("f16", 3, 128), ("bf16", 8, 64)])
def test_store(rt, d, dtype, heads, page):
    """Odd numbers of rows, rows left out, bad rows, strided and unaligned tensors; all else stays."""
    g = torch.Generator().manual_seed(d + heads)
    for n, pad in ((1, 0), (37, 0), (133, 8), (61, 3)):
        pages = -(-2 * n // page) + 1
        t = rt.PageTable(1, pages, page, pages)
        wide = torch.randn(2, n, heads, d + pad, generator=g).to(TYPES[dtype])
        rows = torch.randperm(pages * page, generator=g)[:n].to(torch.int32)
        rows[::5] = -1
        if n > 40:
            rows[3], rows[7] = pages * page, -2
        pools = [torch.randn(pages, heads, page, d, generator=g).to(TYPES[dtype]) for _ in "kv"]
        want = [p.clone() for p in pools]
        for p, x in zip(want, wide[..., pad // 2:pad // 2 + d]):
            for i, at in enumerate(rows.tolist()):
                if 0 <= at < pages * page:
                    p[at // page, :, at % page] = x[i]
        dev = [p.cuda() for p in pools]
        x = wide.cuda()[..., pad // 2:pad // 2 + d]
        t.store(x[0], x[1], rows.cuda(), *dev)
        for got, w in zip(dev, want):
            assert torch.equal(got.cpu(), w)
        assert t.device_error()[1] == (2 if n > 40 else 0)


def test_refusals(rt):
    from accelerator_decode_gb300 import g4
    t = rt.PageTable(2, 4, 16, 2)
    s = i32([0])
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    for call, kind in (
            (lambda: rt.PageTable(2, 4, 24, 2), g4.G4Error), (lambda: rt.PageTable(2, 4, 8, 2), g4.G4Error),
            (lambda: rt.PageTable(2, 0, 16, 2), g4.G4Error), (lambda: rt.PageTable(1025, 4, 16, 2), ValueError),
            (lambda: rt.PageTable(2, 4, 1 << 20, 2), g4.G4Error), (lambda: rt.PageTable(2, 1 << 27, 16, 2), g4.G4Error),
            (lambda: t.extend(i32([0, 1, 0]), i32([1, 1, 1]), 3), g4.G4Error),
            (lambda: t.extend(s, i32([1]), -1), ValueError), (lambda: t.extend(s, i32([1, 2]), 3), ValueError),
            (lambda: t.extend(s.long(), i32([1]), 1), TypeError), (lambda: t.extend(s.cpu(), i32([1]), 1), ValueError),
            (lambda: t.share(s, 2, 1), g4.G4Error), (lambda: t.share(s, 1, 3), g4.G4Error),
            (lambda: t.truncate(s, i32([1, 2])), ValueError),
            (lambda: t.store(k.float(), k, i32([0, 1, 2]), pool, pool), TypeError),
            (lambda: t.store(k, k.half(), i32([0, 1, 2]), pool, pool), TypeError),
            (lambda: t.store(k, k, i32([0, 1]), pool, pool), ValueError),
            (lambda: t.store(k, k, i32([0, 1, 2]), pool[:3], pool), ValueError),
            (lambda: t.store(k[..., :40], k[..., :40], i32([0, 1, 2]), pool, pool), ValueError),
            (lambda: t.store(k.transpose(1, 2), k.transpose(1, 2), i32([0, 1, 2]), pool, pool), ValueError)):
        with pytest.raises(kind):
            call()
    t.store(k[:0], k[:0], i32([]), pool, pool)
    assert t.device_error() == (0, 0)
