"""Numbers that a row does not see leave no trace in it, whatever they are: in front of a sequence, behind it and inside it."""
import math

import pytest

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
