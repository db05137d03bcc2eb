"""Attention over the 4-bit cache where scores are huge: a row goes to its largest score alone, as a
64-bit softmax has it."""
import pytest

import kv4_accuracy as acc

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


def check_one_hot(rt, dtype, d, q_len, scale, grow, kvh=2, group=4, page=0, rising=0.0):
    """Rows times `grow`; the largest score of every output row is far above the next.  rising: keys
    grow by this power of two from row to row as well."""
    n, lens = 2, [150, 67]
    q, k, v = acc.inputs(n, 150, kvh, group, q_len, d, dtype, d + q_len)
    k = k * (2.0 ** (rising * torch.arange(150.0)))[:, None, None].to(k.dtype)
    kw = {}
    if page:
        kw["page_table"] = torch.randperm(20, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(2, 10).cuda()
    c = rt.KV4Cache(n, 150, kvh * group, kvh, d, max_q_len=q_len, page_size=page, track=True, **kw)
    q, order = (q * grow).cuda(), i32([0, 1])
    c.append((k * grow).cuda(), v.cuda(), order, i32([0, 0]), i32(lens))
    rk, rv = c.read(order, i32([0, 0]), 150, i32(lens), dtype=torch.float32)
    out = c.attend(q, order, i32(lens), scale=scale, accumulate=True)
    gained = c.account(order, i32([0, 0]), 150)[1]
    assert c.device_error() == (0, 0)
    for i, ln in enumerate(lens):
        qq = q[i].double().reshape(q_len, kvh, group, d)
        s = torch.einsum("mkgd,tkd->kgmt", qq, rk[i, :ln].double())
        j, last = torch.arange(ln, device="cuda"), ln - q_len + torch.arange(q_len, device="cuda")[:, None]
        s = s.masked_fill(j > last, -float("inf"))
        top = s.topk(2, -1)
        far = (top.values[..., 0] - top.values[..., 1]) * (scale or d ** -0.5)
        # far beyond what rounding the scores can move: 2^-15 of the largest
        sure = far > 1e3 + 2.0 ** -15 * top.values[..., 0].abs() * (scale or d ** -0.5)
        assert sure.float().mean() > 0.9
        hot = top.indices[..., 0]                                                # [kvh, group, m]
        want = torch.stack([rv[i, :ln, h][hot[h]] for h in range(kvh)]).permute(2, 0, 1, 3)  # [m, kvh, group, d]
        got, at = out[i].reshape(q_len, kvh, group, d), sure.permute(2, 0, 1)
        assert torch.equal(got[at], want.to(got.dtype)[at])
        assert out[i].isfinite().all()
        # the account: one for the row that took all, nothing for the others
        sums = gained[i, :, :ln].sum(-1)
        if bool(sure.all()):
            count = torch.zeros(kvh, ln, device="cuda")
            for h in range(kvh):
                count[h].index_add_(0, hot[h].flatten(), torch.ones(hot[h].numel(), device="cuda"))
            assert torch.equal(gained[i, :, :ln], count)
        assert gained[i].isfinite().all() and (sums <= q_len * group * (1 + 1e-6)).all()


@pytest.mark.parametrize("scale", [1e15, 1.1e19, 1e20, 1e30])
@pytest.mark.parametrize("dtype,d,q_len", [("f32", 64, 1), ("bf16", 128, 1), ("f16", 256, 1), ("f32", 512, 1), ("f16", 64, 9),
                                           ("bf16", 64, 20), ("bf16", 128, 64), ("bf16", 256, 33)])
def test_large_scales(rt, dtype, d, q_len, scale):
    check_one_hot(rt, dtype, d, q_len, scale, 1.0)


def test_largest_scale(rt):
    """The largest finite fp32 number, on rows so small that the scores stay in range."""
    check_one_hot(rt, "f32", 64, 1, 3.4028234e38, 2.0 ** -4)
    check_one_hot(rt, "bf16", 128, 20, 3.4028234e38, 2.0 ** -4)


@pytest.mark.parametrize("grow", [2.0 ** 9, 2.0 ** 15, 2.0 ** 20])
@pytest.mark.parametrize("dtype,d,q_len", [("f32", 64, 1), ("bf16", 512, 1), ("bf16", 64, 20), ("bf16", 128, 64), ("bf16", 256, 33)])
def test_large_rows(rt, dtype, d, q_len, grow):
    check_one_hot(rt, dtype, d, q_len, 0.0, grow, page=16)


@pytest.mark.parametrize("rising", [0.1, 0.25, -0.25])
@pytest.mark.parametrize("dtype,d,q_len", [("f32", 256, 1), ("bf16", 512, 1), ("f32", 64, 7), ("bf16", 64, 30), ("bf16", 128, 64),
                                           ("bf16", 256, 33)])
def test_scores_that_grow_and_shrink(rt, dtype, d, q_len, rising):
    """Keys from small to huge, and from huge to small: references are raised past every border."""
    check_one_hot(rt, dtype, d, q_len, 0.0, 2.0 ** 13 if rising > 0 else 2.0 ** 24, page=16, rising=rising)
