"""g4_pages_extend with offsets and new lengths written over its own arguments, and the outputs that it refuses."""
import pytest

import pages_ref as ref

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


def call(rt, t, n, slots, counts, n_rows, rows, offsets, lens):
    return rt._g4.lib.g4_pages_extend(t.h, torch.cuda.current_stream().cuda_stream, n, slots, counts, n_rows, rows, offsets, lens)


@pytest.mark.parametrize("n,each", [(3, 5), (200, 700), (1000, 90)])
def test_over_the_arguments(rt, n, each):
    """Plans of one CTA and of many: all of them read the slots and counts, whoever writes over them."""
    page = 16
    counts = [each - i % 7 for i in range(n)]
    slots = [(i * 7 + 3) % n for i in range(n)] if n % 7 else list(range(n))
    total, most = sum(counts), -(-each // page) + 1
    for round_ in range(5):
        t = rt.PageTable(n, n * most, page, most)
        m = ref.Table(n, n * most, page, most)
        m.holders = lambda p: 1
        a, b, rows = i32(slots + [0]), i32(counts), i32([7] * total)
        assert call(rt, t, n, a.data_ptr(), b.data_ptr(), total, rows.data_ptr(), a.data_ptr(), b.data_ptr()) == 0
        want = m.extend(slots, counts, total)
        assert [rows.tolist(), a.tolist(), b.tolist()] == [list(x) for x in want]
        assert t.table.tolist() == m.table() and t.lens.tolist() == m.lens and t.device_error() == (0, 0)


def test_outputs_that_share_memory(rt):
    t = rt.PageTable(4, 8, 16, 4)
    slots, counts, rows, offsets, lens = i32([0, 1, 0]), i32([3, 4, 0]), i32([9] * 8), i32([9] * 4), i32([9] * 4)
    p = dict(slots=slots.data_ptr(), counts=counts.data_ptr(), rows=rows.data_ptr(), offsets=offsets.data_ptr(), lens=lens.data_ptr())
    for change in (dict(lens=t.lens.data_ptr()), dict(lens=t.lens.data_ptr() + 12), dict(offsets=t.lens.data_ptr()),
                   dict(rows=t.table.data_ptr() + 60), dict(rows=t.lens.data_ptr()), dict(rows=slots.data_ptr()),
                   dict(rows=counts.data_ptr() + 4), dict(rows=offsets.data_ptr()), dict(offsets=rows.data_ptr() + 24),
                   dict(lens=rows.data_ptr() + 24), dict(lens=offsets.data_ptr() + 8)):
        x = {**p, **change}
        assert call(rt, t, 2, x["slots"], x["counts"], 7, x["rows"], x["offsets"], x["lens"]) == -1, change
    assert (t.table == -1).all() and not t.lens.any() and rows.tolist() == [9] * 8 and t.device_error() == (0, 0)
    assert call(rt, t, 2, p["slots"], p["counts"], 7, p["rows"], p["offsets"], p["lens"]) == 0
    assert rows.tolist() == [0, 1, 2, 16, 17, 18, 19, 9] and offsets.tolist() == [0, 3, 7, 9] and lens.tolist() == [3, 4, 9, 9]
