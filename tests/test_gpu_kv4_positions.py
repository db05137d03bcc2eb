"""Positions that g4_kv4_append gives rows by itself: they go on from the newest position that the
slot holds, also after evictions, so that `recent` protects the newest rows."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def rt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from accelerator_decode_gb300 import runtime
    return runtime


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rows(n, m, kvh, d, seed):
    return torch.randn(n, m, kvh, d, generator=torch.Generator().manual_seed(seed)).cuda()


def held(c, slot, n):
    """Positions of a slot's first n rows, [kvh, n]."""
    return c.account(i32([slot]), i32([0]), n)[0][0].cpu().numpy()


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("n,kvh,step", [(3, 2, 1), (3, 1, 5), (40, 3, 61)])
def test_positions_follow_the_tokens(rt, page, n, kvh, step):
    """The loop of a bounded session without positions: a row's position is its token's number, whatever
    was evicted.  Few rows and many (40 x 3 heads x 61 rows go by whole blocks)."""
    d, budget, recent, cap = 64, 70, 9, 70 + 64
    kw = {}
    if page:
        per = -(-cap // page)
        kw["page_table"] = torch.randperm(n * per).to(torch.int32).view(n, per).cuda()
    c = rt.KV4Cache(n, cap, kvh, kvh, d, page_size=page, track=True, **kw)
    g = np.random.default_rng(step)
    slots = i32(g.permutation(n).tolist())
    lens, seen = i32([0] * n), 0
    for turn, m in enumerate([61] + [step] * 20):
        k = rows(n, m, kvh, d, turn)
        w = torch.rand(n, kvh, m, generator=torch.Generator().manual_seed(turn)).cuda()
        c.append(k, k, slots, lens, weights=w)
        lens, seen = lens + m, seen + m
        for i in range(0, n, 13):
            p = held(c, int(slots[i]), int(lens[i]))
            assert (np.sort(p, 1)[:, -min(m, seen):] == np.arange(seen - m, seen)).all()
            np.testing.assert_array_equal(p[:, -m:], np.tile(np.arange(seen - m, seen), (kvh, 1)))
            assert all(len(set(x)) == len(x) for x in p)
        lens = c.evict(slots, lens, budget, recent)
        for i in range(0, n, 13):
            p = held(c, int(slots[i]), int(lens[i]))
            assert set(range(seen - min(recent, seen), seen)) <= set(p[0].tolist()) & set(p[-1].tolist())
    assert c.device_error() == (0, 0)


def test_slots_begin_anew_and_given_positions_are_carried_on(rt):
    d, kvh = 64, 2
    c = rt.KV4Cache(3, 64, kvh, kvh, d, track=True)
    k = rows(3, 20, kvh, d, 1)
    c.append(k, k, i32([0, 1, 2]), i32([0, 0, 0]))
    assert c.evict(i32([0, 1]), i32([20, 20]), 8, 4).tolist() == [8, 8]
    c.append(k[:, :3], k[:, :3], i32([0, 1, 2]), i32([8, 0, 20]))
    assert held(c, 0, 11)[:, 8:].tolist() == [[20, 21, 22]] * kvh         # cut: on from the newest
    assert held(c, 1, 3).tolist() == [[0, 1, 2]] * kvh                    # begun anew
    assert held(c, 2, 23).tolist() == [list(range(23))] * kvh             # never cut: the row
    c.append(k[:, :2], k[:, :2], i32([0, 1, 2]), i32([11, 3, 23]), counts=i32([2, 0, 2]))
    assert held(c, 0, 13)[:, 11:].tolist() == [[23, 24]] * kvh
    # nothing appended at row 0 begins nothing
    c.append(k[:1, :1], k[:1, :1], i32([0]), i32([0]), counts=i32([0]))
    c.append(k[:1, :1], k[:1, :1], i32([0]), i32([13]))
    assert held(c, 0, 14)[:, 13].tolist() == [25, 25]
    # a slot put back with its positions, out of order as an eviction leaves them, per head
    pos = torch.stack([torch.randperm(20) * 3 + 5, torch.randperm(20) + 900]).to(torch.int32).cuda()[None].contiguous()
    c.append(k[:1], k[:1], i32([1]), i32([0]), positions=pos)
    c.append(k[:1, :2], k[:1, :2], i32([1]), i32([20]))
    now = held(c, 1, 22)
    np.testing.assert_array_equal(now[:, :20], pos[0].cpu().numpy())
    assert (now[:, 20] > now[:, :20].max(1)).all() and (now[:, 21] == now[:, 20] + 1).all()
    rising = torch.arange(100, 120, dtype=torch.int32, device="cuda").expand(1, kvh, 20).contiguous()
    c.append(k[:1], k[:1], i32([2]), i32([0]), positions=rising)
    c.append(k[:1, :2], k[:1, :2], i32([2]), i32([20]))
    assert held(c, 2, 22)[:, 20:].tolist() == [[120, 121]] * kvh
    assert c.evict(i32([2]), i32([22]), 10, 3).tolist() == [10]
    c.append(k[:1, :2], k[:1, :2], i32([2]), i32([10]))
    assert held(c, 2, 12)[:, 10:].tolist() == [[122, 123]] * kvh
    # the largest positions there are: no wrap below the rows that are there
    top = torch.arange(2 ** 31 - 21, 2 ** 31 - 1, dtype=torch.int64).to(torch.int32).cuda().expand(1, kvh, 20).contiguous()
    c.append(k[:1], k[:1], i32([0]), i32([0]), positions=top)
    c.append(k[:1, :3], k[:1, :3], i32([0]), i32([20]))
    assert held(c, 0, 23)[:, 20:].tolist() == [[2 ** 31 - 1] * 3] * kvh
    assert c.device_error() == (0, 0)


def test_positions_in_a_graph(rt):
    """A captured step of append, attend and evict: every replay's token has the next position."""
    d, n, budget = 128, 2, 40
    c = rt.KV4Cache(n, budget + 1, 8, 1, d, max_q_len=1, track=True)
    k, q = rows(n, budget, 1, d, 1), rows(n, 1, 8, d, 2)
    slots, start, lens = i32([1, 0]), i32([budget] * n), i32([budget + 1] * n)
    c.append(k, k, slots, i32([0, 0]))
    k1 = rows(n, 1, 1, d, 3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.append(k1, k1, slots, start)
        c.attend(q, slots, lens, accumulate=True)
        c.evict(slots, lens, budget, 6)
    for i in range(9):
        graph.replay()
    for s in range(n):
        p = held(c, s, budget)[0]
        assert set(range(budget + 3, budget + 9)) <= set(p.tolist()) and p.max() == budget + 8
        assert len(set(p.tolist())) == budget
    assert c.device_error() == (0, 0)


def test_recent_rows_stay_recent(rt):
    """A slot put back out of order goes on with the next position, not a later one, so that the rows
    that were recent still are; evictions one after the other do not step back."""
    d, kvh = 64, 2
    c = rt.KV4Cache(2, 64, kvh, kvh, d, track=True)
    k = rows(1, 40, kvh, d, 1)
    order = torch.stack([torch.randperm(30, generator=torch.Generator().manual_seed(h)) for h in range(kvh)])
    at = int((order[0] == 29).nonzero())
    order[0, at], order[0, 0] = int(order[0, 0]), 29                # the newest at row 0
    pos = order.to(torch.int32).cuda()[None].contiguous()
    for cuts in ((0, 30), (0, 11, 30), (0, 1, 2, 30)):                                   # in one call, in several
        for a, b in zip(cuts, cuts[1:]):
            c.append(k[:, a:b], k[:, a:b], i32([1]), i32([a]), positions=pos[:, :, a:b].contiguous())
        c.append(k[:, :1], k[:, :1], i32([1]), i32([30]))
        assert held(c, 1, 31)[:, 30].tolist() == [30, 30], cuts
    assert c.evict(i32([1]), i32([31]), 12, 12).tolist() == [12]
    assert np.sort(held(c, 1, 12), 1).tolist() == [list(range(19, 31))] * kvh
    # the newest rows go by weight (recent 0): their positions are not given again
    w = torch.ones(1, kvh, 20, device="cuda")
    w[..., 15:] = 0
    c.append(k[:, :20], k[:, :20], i32([0]), i32([0]), weights=w)
    assert c.evict(i32([0]), i32([20]), 15, 0).tolist() == [15]
    assert c.evict(i32([0]), i32([15]), 10, 0).tolist() == [10]
    c.append(k[:, :2], k[:, :2], i32([0]), i32([10]))
    assert held(c, 0, 12).tolist() == [list(range(10)) + [20, 21]] * kvh
    # rows that the caller takes back (refused drafts) give their positions back
    c.append(k[:, :5], k[:, :5], i32([0]), i32([12]))
    c.append(k[:, :1], k[:, :1], i32([0]), i32([13]))
    assert held(c, 0, 14)[:, 12:].tolist() == [[22, 23]] * kvh
    assert c.device_error() == (0, 0)


def test_more_rows_at_recent_positions_than_the_budget(rt):
    """Positions that rows share: the lowest rows stay, whatever their weights."""
    d = 64
    c = rt.KV4Cache(1, 40, 1, 1, d, track=True)
    k = rows(1, 40, 1, d, 1)
    pos = torch.zeros(1, 1, 40, dtype=torch.int32, device="cuda")
    pos[..., 5:] = 9
    pos[..., 38:] = 8
    w = torch.rand(1, 1, 40, generator=torch.Generator().manual_seed(1)).cuda()
    c.append(k, k, i32([0]), i32([0]), positions=pos, weights=w)
    before = c.read(i32([0]), i32([0]), 40, dtype=torch.float32)[0]
    assert c.evict(i32([0]), i32([40]), 7, 2).tolist() == [7]
    p, gw = c.account(i32([0]), i32([0]), 7)
    kept = [7, 8, 9, 10, 11, 5, 6]               # rows 5 and 6 stay in place, 7 .. 11 fill rows 0 .. 4
    assert (p == 9).all() and torch.equal(gw[0, 0], w[0, 0, kept])
    assert torch.equal(c.read(i32([0]), i32([0]), 7, dtype=torch.float32)[0][0], before[0, kept])
    assert c.device_error() == (0, 0)
