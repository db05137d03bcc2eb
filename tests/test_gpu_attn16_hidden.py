"""Numbers that a row does not see leave no trace in it, whatever they are: in front of a sequence, behind it and inside it."""
import math

import pytest

import kv4_accuracy as acc

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


def rows(n, heads, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, heads, d, generator=g).to(TYPES[dtype]).cuda()


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype,heads,kvh", [("bf16", 8, 1), ("f16", 6, 2), ("bf16", 64, 1)])
@pytest.mark.parametrize("window", [0, 70])
def test_rows_behind_a_sequence(rt, d, dtype, heads, kvh, window):
    """Rows of no sequence between and behind the sequences' last tiles: zeros or NaN, the same bits.  Lengths a few tokens
    past a tile, so that several blocks of rows end before their sequence does and their last tile behind it."""
    lens, gap = [129 + 40, 3, 257], 140
    n, spans, at = sum(lens) + gap * len(lens), [], 0
    q, k, v = rows(n, heads, d, dtype, d), rows(n, kvh, d, dtype, d + 1), rows(n, kvh, d, dtype, d + 2)
    hole = torch.ones(n, dtype=torch.bool)
    for m in lens:
        spans.append((at, at + m))
        hole[at:at + m] = False
        at += m + gap
    a = rt.Attention(heads, kvh, d, dtype=TYPES[dtype], max_seqs=1)
    got = []
    for fill in (0.0, math.nan, math.inf):
        for x in (q, k, v):
            x[hole.cuda()] = fill
        got.append([a.prompt(q, k, v, i32([x, y]), window=window)[x:y] for x, y in spans])
    assert a.device_error() == (0, 0)
    for other in got[1:]:
        for x, y in zip(got[0], other):
            assert torch.isfinite(x).all() and torch.equal(x, y)


@pytest.mark.parametrize("d,heads,kvh,t,window", [(64, 6, 2, 9001, 0), (128, 8, 2, 16400, 0), (256, 8, 1, 6001, 0), (256, 8, 1, 6001, 512),
                                                  (512, 8, 1, 16400, 0), (512, 3, 3, 3333, 700)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_values_hidden_inside_a_long_sequence(rt, d, heads, kvh, t, window, dtype):
    """A row of NaN and single infinities near the end: rows in front of them (and behind the window) are right, the rows that
    see them are not finite in those columns, and the call ends in time.

    An output row is off by its own rounding, at most u of it, where its weights are 32-bit ones, or by 1.3 u where they
    go into a product in 16 bits (test_gpu_attn16); 32-bit scores, exponentials and sums add d / 16 steps of 2^-21 after the scale,
    2^-22, and 2^-23 a step of keys / 16 + 32.
    128 rows of a block, four at a time by each of four warps, are 8 times t / 4 steps of about 1,500 cycles: 26 ms at
    16,400; ten times that is allowed."""
    q, k, v = rows(t, heads, d, dtype, d + t), rows(t, kvh, d, dtype, 1), rows(t, kvh, d, dtype, 2)
    clean = v.clone()
    nan_at, inf_at = t - 400, t - 70
    v[nan_at, 0] = math.nan
    v[inf_at, kvh - 1, 5], v[inf_at + 3, kvh - 1, d - 1] = math.inf, -math.inf
    off = i32([0, t])
    a = rt.Attention(heads, kvh, d, dtype=TYPES[dtype], max_seqs=1)
    a.prompt(q, k, clean, off, window=window)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    out = a.prompt(q, k, v, off, window=window)
    end.record()
    assert a.device_error() == (0, 0)
    assert begin.elapsed_time(end) < 260
    x = t - 700                                             # some tiles around and in front of them
    want = acc.attend(q[x:], k, clean, None, window)[0].reshape(t - x, heads, d)
    keys = window or t
    u = torch.finfo(TYPES[dtype]).eps / 2
    lim = 1.3 * u + d / 16 * 2.0 ** -21 + 2.0 ** -22 + (keys / 16 + 32) * 2.0 ** -23 + (4 * 2.0 ** -25 * math.sqrt(keys) if dtype == "f16" else 0)
    bad = torch.zeros(t, kvh, d, dtype=torch.bool, device="cuda")
    for i in range(t - 700, t):                             # columns that row i sees a number in that is not finite
        first = max(0, i - window + 1) if window else 0
        bad[i] = ~torch.isfinite(v[max(first, t - 700):i + 1]).all(0)
    bad = bad[x:].repeat_interleave(heads // kvh, 1)
    got = out[x:].double()
    assert not torch.isfinite(got[bad]).any() and torch.isfinite(got[~bad]).all()
    diff, ref = torch.where(bad, 0.0, got - want), torch.where(bad, 0.0, want)
    whole = ~bad.all(-1)
    err = (diff.norm(dim=-1) / ref.norm(dim=-1))[whole]
    assert float(err.max()) <= lim, (float(err.max()), lim)
    assert torch.equal(out.nan_to_num(7.0), a.prompt(q, k, v, off, window=window).nan_to_num(7.0))


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("many", [0, 100])
def test_rows_of_no_sequence_where_offsets_fall(rt, d, many):
    """A new result is zero in front of every sequence that is attended to and behind every one, and their own rows are
    right, although the first offset is not the lowest or the last not the highest."""
    n, heads, kvh = 400, 4, 2
    q, k, v = rows(n, heads, d, "bf16", d), rows(n, kvh, d, "bf16", 1), rows(n, kvh, d, "bf16", 2)
    a = rt.Attention(heads, kvh, d, max_seqs=4 + many)
    for offsets, good in (([0, 300, 10], [(0, 300)]), ([300, 5, 350], [(5, 350)]), ([390, 20, 200, 100, 100], [(20, 200)]),
                          ([0, 300, 300, 300, 7], [(0, 300)]), ([1000, 40, 60, 3], [(40, 60)])):
        offsets = offsets[:-1] + [offsets[-2]] * many + offsets[-1:]
        for _ in range(20):
            out = a.prompt(q, k, v, i32(offsets))
            assert a.device_error() == (-7, 2)
            clamped = [min(max(x, 0), n) for x in (offsets[0], offsets[-1])]
            front, end = min([clamped[0]] + [x for x, _ in good]), max([max(clamped)] + [y for _, y in good])
            assert not out[:front].any() and not out[end:].any()
            for x, y in good:
                want, _ = acc.attend(q[x:y], k[x:y], v[x:y])
                err = acc.row_errors(out[x:y], want).max()
                assert err <= 2.5 * 2.0 ** -8 + d / 16 * 2.0 ** -21 + 2.0 ** -22 + 64 * 2.0 ** -23
