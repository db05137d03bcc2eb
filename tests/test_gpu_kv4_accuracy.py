"""The 4-bit cache's attention and account on the GPU against 64 bits, within the errors that
kv4_accuracy derives (a host test shows that wrong results are outside them)."""
import math

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


def filled(rt, lens, kvh, group, q_len, d, dtype, page=0, track=False, seed=0):
    """A cache of the sequences' rows, the queries, and the values the rows stand for."""
    n, keys = len(lens), max(max(lens), 1)
    kw = {}
    if page:
        per = -(-keys // page)
        order = torch.randperm(n * per, generator=torch.Generator().manual_seed(seed + 5))
        kw["page_table"] = order.to(torch.int32).view(n, per).cuda()
    c = rt.KV4Cache(n, keys, kvh * group, kvh, d, max_q_len=q_len, page_size=page, track=track, **kw)
    q, k, v = (x.cuda() for x in acc.inputs(n, keys, kvh, group, q_len, d, dtype, seed))
    order = i32(list(range(n)))
    c.append(k, v, order, i32([0] * n), i32(lens))
    return c, q, order, c.read(order, i32([0] * n), keys, i32(lens), dtype=torch.float32)


def compare(c, q, order, rows, lens, dtype, d, window=0, track=False, q_lens=None, few=False):
    q_len = q.shape[1]
    out = c.attend(q, order, i32(lens), None if q_lens is None else i32(q_lens), window=window, accumulate=track)
    gained = c.account(order, i32([0] * len(lens)), rows[0].shape[1])[1] if track else None
    for i, ln in enumerate(lens):
        m = q_len if q_lens is None else q_lens[i]
        want, gain = acc.attend(q[i, :m], rows[0][i, :ln], rows[1][i, :ln], window=window)
        worst = float(acc.row_errors(out[i, :m], want).max()) if m else 0.0
        assert acc.right(out[i, :m], want, dtype, ln, few), (i, ln, worst, acc.row_limit(dtype, d, ln, few))
        assert not out[i, m:].any()
        if track:
            off = float(((gained[i, :, :ln].double() - gain).norm(dim=-1) / gain.norm(dim=-1)).max())
            assert acc.gains_right(gained[i, :, :ln], gain, dtype, d), (i, ln, off, acc.gain_limit(dtype, d))
    assert c.device_error() == (0, 0)


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kvh,group,page,track", [(1, 8, 0, True), (2, 3, 128, False), (1, 20, 16, True)])
def test_single_tokens(rt, d, dtype, kvh, group, page, track):
    lens = [1, 16, 200, 700, 4099, 65]
    c, q, order, rows = filled(rt, lens, kvh, group, 1, d, dtype, page, track, d + group)
    compare(c, q, order, rows, lens, dtype, d, track=track)


@pytest.mark.parametrize("d", [64, 256, 512])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_many_sequences(rt, d, dtype):
    """More items than CTAs: whole items, and spans that end inside one."""
    lens = [(i * 977) % 1465 + 1 for i in range(120)]
    c, q, order, rows = filled(rt, lens, 1, 8, 1, d, dtype, 64, True, d)
    compare(c, q, order, rows, lens, dtype, d, track=True)


@pytest.mark.parametrize("d,dtype", [(256, "bf16"), (512, "f32"), (128, "f16")])
def test_long_context(rt, d, dtype):
    lens = [30011, 5, 20000]
    c, q, order, rows = filled(rt, lens, 1, 8, 1, d, dtype, 128, True, 7)
    compare(c, q, order, rows, lens, dtype, d, track=True)


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("q_len,kvh,group,page", [(7, 4, 3, 16), (64, 1, 8, 0), (33, 2, 1, 128)])
def test_token_blocks(rt, d, dtype, q_len, kvh, group, page):
    lens = [q_len, 700, 130, 2051, 0, 1, 65]
    q_lens = [q_len, q_len, max(1, q_len // 2), q_len, q_len, 1, 0]
    c, q, order, rows = filled(rt, lens, kvh, group, q_len, d, dtype, page, True, d + q_len)
    compare(c, q, order, rows, lens, dtype, d, track=True, q_lens=q_lens)


@pytest.mark.parametrize("window", [1, 63, 64, 300])
@pytest.mark.parametrize("d,dtype,q_len,group", [(64, "f32", 1, 8), (512, "f16", 1, 8), (128, "bf16", 9, 8), (256, "bf16", 1, 8)])
def test_windows(rt, window, d, dtype, q_len, group):
    lens = [q_len, 64, 65, 900, 40]
    c, q, order, rows = filled(rt, lens, 2, group, q_len, d, dtype, 32, False, window)
    compare(c, q, order, rows, lens, dtype, d, window=window)


# ------------------------------------------------------------------------- the kept bits
@pytest.mark.parametrize("dtype,low", [("f32", 20), ("f16", 10)])
@pytest.mark.parametrize("d", [64, 512])
def test_every_bit_of_a_query_counts(rt, dtype, low, d):
    """Queries A + r 2^-low whose A cancels: rows of a key hold +a and -a side by side, so the scores
    are sums of a (r - r') 2^-low, small whole numbers after a scale of 2^low / 64.  fp32 queries have
    A = 1 + s 2^-9 and so need all 24 bits."""
    g = torch.Generator().manual_seed(d)
    t, heads = 200, 8
    a = torch.randint(-7, 8, (1, t, 1, d // 2), generator=g).float()
    a[..., ::16] = 7                                               # every group has a scale of one
    k = torch.stack([a, -a], -1).flatten(-2)
    s = torch.randint(0, 512, (1, 1, heads, d // 2, 1), generator=g) if dtype == "f32" else torch.zeros(1, 1, heads, d // 2, 1)
    r = torch.randint(0, 8 if d == 64 else 4, (1, 1, heads, d // 2, 2), generator=g)
    q = (1 + s.double() * 2.0 ** -9 + r.double() * 2.0 ** -low).flatten(-2)
    assert torch.equal(q.to(acc.TYPES[dtype]).double(), q)
    v = torch.randn(1, t, 1, d, generator=g)
    c = rt.KV4Cache(1, t, heads, 1, d, max_q_len=1)
    c.append(k.cuda(), v.cuda(), i32([0]), i32([0]))
    rk, rv = c.read(i32([0]), i32([0]), t, dtype=torch.float32)
    assert torch.equal(rk.cpu(), k)
    scale = 2.0 ** low / 64
    out = c.attend(q.to(acc.TYPES[dtype]).cuda(), i32([0]), i32([t]), scale=scale)
    want, _ = acc.attend(q[0].cuda(), rk[0], rv[0], scale=scale)
    assert acc.right(out[0], want, dtype, t), float(acc.row_errors(out[0], want).max())
    # one bit less, and the result is another: the check above sees it
    less = (q * 2.0 ** (low - 1)).round() * 2.0 ** (1 - low)
    assert not acc.right(acc.attend(less[0].cuda(), rk[0], rv[0], scale=scale)[0].to(acc.TYPES[dtype]), want, dtype, t)


def test_weights_of_fp32_calls_keep_24_bits(rt):
    """Values +1 and -1 under weights p and p (1 + 2^-14), with a third row as the maximum: the output
    is p 2^-14, so a weight cut to 16 bits (2^-18 of p) is off by a sixteenth of it.  What may be off:
    the exponentials' 2^-22 each, and 2^-24 of scores below 16, both against 2^-14: 2^-7 together."""
    heads, d = 8, 64
    delta = math.log1p(2.0 ** -14)
    base = torch.linspace(-0.3, -2.4, heads).double()              # scores of the two rows, per head
    q = torch.zeros(1, 1, heads, d)
    q[0, 0, :, 0] = base.float()
    q[0, 0, :, 32] = delta
    k = torch.zeros(1, 3, 1, d)
    k[0, 1, 0, 0] = k[0, 2, 0, 0] = 7.0                            # 7 under a scale of one; row 0 scores 0
    k[0, 2, 0, 32] = 7.0
    v = torch.zeros(1, 3, 1, d)
    v[0, 1], v[0, 2] = -7.0, 7.0
    c = rt.KV4Cache(1, 3, heads, 1, d, max_q_len=1)
    c.append(k.cuda(), v.cuda(), i32([0]), i32([0]))
    out = c.attend(q.cuda(), i32([0]), i32([3]), scale=1.0 / 7).cpu().double()[0]
    want, _ = acc.attend(q[0], k[0], v[0], scale=1.0 / 7)
    assert (want.abs() > 2.0 ** -17).all()
    assert (out - want).norm() <= 2.0 ** -5 * want.norm(), float((out - want).norm() / want.norm())


# ------------------------------------------------- paths that only some calls take
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,q_len,track", [(64, 1, True), (128, 64, True), (256, 64, True), (64, 33, False), (512, 1, True), (256, 9, False)])
def test_scales_outside_the_narrow_range(rt, dtype, d, q_len, track):
    """Rows with scales beyond [2^-60, 2^57] are decoded the plain way: keys whose first 32 numbers are
    2^62 times larger (and the queries' as much smaller), values whose last 32 are 2^-70 of the others."""
    lens, group = [700, 65, 130], 8
    n, keys = len(lens), 700
    q, k, v = acc.inputs(n, keys, 1, group, q_len, d, dtype, d + q_len)
    k[..., :32] *= 2.0 ** 62
    q[..., :32] *= 2.0 ** -62
    v[..., -32:] *= 2.0 ** -70
    c = rt.KV4Cache(n, keys, group, 1, d, max_q_len=q_len, track=track)
    q, order = q.cuda(), i32([0, 1, 2])
    c.append(k.cuda(), v.cuda(), order, i32([0] * n), i32(lens))
    rows = c.read(order, i32([0] * n), keys, i32(lens), dtype=torch.float32)
    # (half of a row's numbers or less make up its norm: 32 at d = 64)
    compare(c, q, order, rows, lens, dtype, d, track=track, few=True)
    out = c.attend(q, order, i32(lens)).double()
    for i, ln in enumerate(lens):                                  # the tiny numbers by themselves
        want, _ = acc.attend(q[i], rows[0][i, :ln], rows[1][i, :ln])
        assert bool((acc.row_errors(out[i, ..., -32:], want[..., -32:]) <= acc.row_limit(dtype, d, ln, few=True)).all())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("track", [False, True])
def test_blocks_of_strided_tokens(rt, d, track):
    """Queries and outputs of token blocks as slices of packed, shifted and broadcast tensors: equal to
    the dense call's, bit by bit, and nothing beside the output is written."""
    n, t, m, kvh, group = 2, 150, 20, 2, 4
    heads = kvh * group
    lens, order = [t, 77], i32([0, 1])

    def fresh():
        return filled(rt, lens, kvh, group, m, d, "bf16", 16, track, 3)

    c, q, _, _ = fresh()
    want = c.attend(q, order, i32(lens), accumulate=track)
    gained = c.account(order, i32([0, 0]), t)[1] if track else None
    for shift, pad in ((0, 8), (8, 8), (8, 16), (4, 4), (1, 5)):   # 16-byte, 32-byte, 8-byte, odd places
        c, _, _, _ = fresh()
        pack = torch.full((n, heads, m, d + pad + shift), 9.0, dtype=torch.bfloat16, device="cuda")
        src = pack.transpose(1, 2)[..., shift:shift + d]
        src.copy_(q)
        buf = torch.full((n, m, heads, d + pad + shift), 7.0, dtype=torch.bfloat16, device="cuda")
        dst = buf[..., shift:shift + d]
        assert c.attend(src, order, i32(lens), accumulate=track, out=dst) is dst
        assert torch.equal(dst, want), (shift, pad)
        assert (buf[..., :shift] == 7).all() and (buf[..., shift + d:] == 7).all()
        if track:
            assert torch.equal(c.account(order, i32([0, 0]), t)[1], gained)
        c.close()
    one = q[:, :1].expand(n, m, heads, d)
    assert torch.equal(c_attend(fresh, one, order, lens), c_attend(fresh, one.contiguous(), order, lens))


def c_attend(fresh, q, order, lens):
    c, _, _, _ = fresh()
    return c.attend(q, order, i32(lens))


@pytest.mark.parametrize("d,rows", [(64, 96), (64, 98), (128, 64), (128, 66), (256, 48), (256, 50)])
@pytest.mark.parametrize("tokens", [True, False])
def test_both_sides_of_the_block_kernels_border(rt, d, rows, tokens):
    """The most query rows per KV head that the single-token path takes, and two more: as tokens of one
    head, and as heads of as few tokens as there can be."""
    q_len = rows if tokens else -(-rows // 64)
    while rows % q_len or q_len > 64:
        q_len = q_len - 1 if tokens else q_len + 1
    group = rows // q_len
    lens = [q_len, 700, 65, 2051]
    c, q, order, kv = filled(rt, lens, 2, group, q_len, d, "bf16", 64, True, rows)
    compare(c, q, order, kv, lens, "bf16", d, track=True)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_strided_blocks_of_128_rows(rt, d):
    """Odd and 8-byte places once more, with rows enough for the block kernels at every width."""
    n, t, m, heads, lens, order = 2, 150, 32, 4, [150, 77], i32([0, 1])
    fresh = lambda: filled(rt, lens, 1, heads, m, d, "bf16", 16, True, 4)
    c, q, _, _ = fresh()
    want = c.attend(q, order, i32(lens), accumulate=True)
    gained = c.account(order, i32([0, 0]), t)[1]
    for shift, pad in ((8, 8), (4, 4), (1, 5)):
        c, _, _, _ = fresh()
        src = torch.full((n, heads, m, d + pad + shift), 9.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)[..., shift:shift + d]
        src.copy_(q)
        buf = torch.full((n, m, heads, d + pad + shift), 7.0, dtype=torch.bfloat16, device="cuda")
        c.attend(src, order, i32(lens), accumulate=True, out=buf[..., shift:shift + d])
        assert torch.equal(buf[..., shift:shift + d], want)
        assert (buf[..., :shift] == 7).all() and (buf[..., shift + d:] == 7).all()
        assert torch.equal(c.account(order, i32([0, 0]), t)[1], gained)


def test_not_finite_query_stays_in_its_row_of_a_block(rt):
    d, t, m = 128, 100, 16
    c, q, order, _ = filled(rt, [t], 1, 8, m, d, "bf16", 0, False, 5)
    clean = c.attend(q, order, i32([t]))
    q[0, 1, 3, 5], q[0, 0, 6, 0], q[0, 15, 7, 9] = float("nan"), float("inf"), float("-inf")
    out = c.attend(q, order, i32([t]))
    bad = torch.zeros(m, 8, dtype=torch.bool, device="cuda")
    bad[1, 3] = bad[0, 6] = bad[15, 7] = True
    assert out[0][bad].isnan().all() and torch.equal(out[0][~bad], clean[0][~bad])


def test_more_sequences_than_the_block_kernels_hold(rt):
    """Token blocks of 400 sequences: their spans do not fit beside a block kernel's operands."""
    lens = [13 + (i * 37) % 60 for i in range(400)]
    c, q, order, rows = filled(rt, lens, 1, 8, 13, 64, "bf16", 16, True, 9)
    compare(c, q, order, rows, lens, "bf16", 64, track=True)
