"""Attention over 16-bit keys and values where a CTA takes many items, one after the other: barriers, rings and results go
from one to the next.  And the weights of rows that each sequence reads on its own, in two bf16 parts."""
import pytest

import kv4_accuracy as acc
from test_gpu_attn16 import check_prompt, check_shared, pool_of

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


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("t", [300, 60])
def test_rising_scores_of_many_items(rt, d, dtype, t):
    """Hundreds of sequences alike, whose references are raised in every tile: the same bits for all, and the right ones."""
    n = 400
    q = torch.zeros(t, 2, d)
    q[:, :, 0] = 4.0
    k = torch.zeros(t, 1, d)
    k[:, 0, 0] = torch.arange(t) * 0.5
    v = torch.randn(t, 1, d, generator=torch.Generator().manual_seed(1))
    q, k, v = (x.to(TYPES[dtype]).cuda() for x in (q, k, v))
    a = rt.Attention(2, 1, d, dtype=TYPES[dtype], max_seqs=n)
    offsets = i32([t * i for i in range(n + 1)])
    for keys, values in ((k, v), (k.flip(0), v)):
        out = a.prompt(q.repeat(n, 1, 1), keys.repeat(n, 1, 1), values.repeat(n, 1, 1), offsets, scale=1.0).view(n, t, 2, d)
        assert a.device_error() == (0, 0)
        check_prompt(out[0], q, keys, values, [0, t], dtype, scale=1.0)
        assert (out == out[:1]).all()


# more items than SMs, whole prefixes each; and prefixes long enough that their parts take all SMs
@pytest.mark.parametrize("d,heads,kvh,n,rows", [(128, 256, 16, 200, 1152), (64, 256, 16, 200, 2176), (256, 256, 16, 96, 1152),
                                                (512, 128, 8, 96, 1152), (64, 128, 8, 96, 8192), (256, 128, 8, 96, 4096),
                                                (512, 128, 8, 96, 1664)])
def test_many_items_of_a_prefix(rt, d, heads, kvh, n, rows):
    page = 64
    lens = [0 if i % 13 == 5 else rows + (37 * i * i) % 60 if i % 7 else rows for i in range(n)]
    t, pools, dense = pool_of(rt, lens, rows // page, kvh, d, "bf16", page, d + n)
    a = rt.Attention(heads, kvh, d, max_seqs=n)
    q, out = check_shared(rt, a, t, pools, dense, rows // page, heads, kvh, d, "bf16", seed=heads)
    for _ in range(3):
        assert torch.equal(out, a.shared(q, *pools, t, i32(list(range(n))), rows // page))


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("shared", [0, 4])
def test_two_parts_of_a_weight(rt, d, shared):
    """Weights in two bf16 parts are off by 2^-17 of themselves: in the mean over many rows, a result is off as the 64-bit
    one rounded once is, and by 32-bit scores (d / 16 steps of 2^-21 after the scale), exponentials (2^-22) and sums (2^-23 for each
    of keys / 16 + 32 steps).  One part, off by 0.4 of 2^-8 in the mean as the result's own rounding is, would give 1.3
    times as much or more."""
    heads, kvh, page, n = 16, 2, 16, 24
    lens = [shared * page + 150 + 9 * i for i in range(n)]
    t, pools, dense = pool_of(rt, lens, shared, kvh, d, "bf16", page, d)
    a = rt.Attention(heads, kvh, d, max_seqs=n)
    q = torch.randn(n, heads, d, generator=torch.Generator().manual_seed(d)).bfloat16().cuda()
    out = a.shared(q, *pools, t, i32(list(range(n))), shared)
    assert a.device_error() == (0, 0)
    want = torch.cat([acc.attend(q[i:i + 1], *dense[i])[0] for i in range(n)])
    once = acc.row_errors(want.bfloat16(), want).mean()
    more = 2.0 ** -17 + d / 16 * 2.0 ** -21 + 2.0 ** -22 + (max(lens) / 16 + 32) * 2.0 ** -23
    assert acc.row_errors(out, want).mean() <= once + more
