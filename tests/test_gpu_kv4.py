"""The 4-bit KV cache on the GPU against a plain 64-bit implementation (kv4_ref).

What is stored is compared for equality.  The attention's bound is worked out from its
arithmetic in `attend_bound`."""
import numpy as np
import pytest

import kv4_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def rt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from accelerator_decode_gb300 import runtime
    return runtime


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def host(t):
    return t.detach().cpu().double().numpy()


def make(rt, n_slots, capacity, heads, kvh, d, page=0, seed=0, **kw):
    if page:
        per = -(-capacity // page)
        g = torch.Generator().manual_seed(seed + 17)
        kw.setdefault("page_table", torch.randperm(n_slots * per + 3, generator=g)[:n_slots * per].to(torch.int32)
                      .view(n_slots, per).cuda())
        kw.setdefault("n_pages", n_slots * per + 3)
    return rt.KV4Cache(n_slots, capacity, heads, kvh, d, page_size=page, **kw)


def rows(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp(torch.randn(*shape[:-1], 1, generator=g))
    x[..., ::37] *= 5
    return x.to(TYPES[dtype]).cuda()


def fine(cache):
    assert cache.device_error() == (0, 0)


# ------------------------------------------------------------------------------ rows
@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("page", [0, 16, 64])
def test_append_read(rt, d, dtype, page):
    """Odd row counts from odd places, three heads, slots out of order; other rows untouched."""
    n, kvh, m = 3, 3, 37
    c = make(rt, 5, 131, 6, kvh, d, page)
    k, v = rows((n, m, kvh, d), dtype, 1), rows((n, m, kvh, d), dtype, 2)
    slots, start, counts = i32([3, 0, 4]), i32([5, 0, 94]), i32([37, 0, 11])
    c.append(k, v, slots, start, counts)
    for typ in TYPES.values():
        rk, rv = c.read(slots, start, m, counts, dtype=typ)
        for got, x in ((rk, k), (rv, v)):
            want = ref.values(host(x))
            for i, cnt in enumerate([37, 0, 11]):
                w = torch.from_numpy(want[i, :cnt]).to(typ).double().numpy()
                np.testing.assert_array_equal(host(got[i, :cnt]), w)
                assert not host(got[i, cnt:]).any()
    allk, allv = c.read(i32([3]), i32([0]), 131)
    assert not host(allk[:, :5]).any() and not host(allk[:, 42:]).any() and not host(allv[:, 42:]).any()
    fine(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_append_strided_unaligned(rt, dtype):
    """Transposed heads, odd strides and bases that are not 16-byte aligned; a broadcast value."""
    n, m, kvh, d = 2, 9, 2, 64
    big = rows((n, kvh, m, d + 3), dtype, 3)
    k = big.transpose(1, 2)[..., 1:1 + d]
    v = rows((1, 1, 1, d), dtype, 4).expand(n, m, kvh, d)
    c = make(rt, 2, 20, 2, kvh, d)
    c.append(k, v, i32([1, 0]), i32([3, 11]))
    rk, rv = c.read(i32([1, 0]), i32([3, 11]), m)
    np.testing.assert_array_equal(host(rk), ref.values(host(k)))
    np.testing.assert_array_equal(host(rv), ref.values(host(v)))
    fine(c)


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("page,pad", [(0, 0), (16, 3), (64, 8)])
def test_append_read_many(rt, d, dtype, page, pad):
    """Calls large enough to go by whole blocks of rows: ragged starts and counts, blocks filled by
    two calls, ties (multiples of half a step), NaN and infinities, a missing page, rows kept."""
    n, kvh, m, cap = 44, 3, 61, 131                   # 44 sequences x 3 heads x 4 blocks
    g = np.random.default_rng(d + page)
    c = make(rt, n + 1, cap, 3, kvh, d, page)
    a, b = (rows((n, m, kvh, d + pad), dtype, s)[..., pad // 2:pad // 2 + d] for s in (1, 2))
    a[::3, :, :, :32] = torch.randint(-14, 15, (15, m, kvh, 32), generator=torch.Generator().manual_seed(3)).to(a) * 0.5
    a[::3, :, :, 5] = 7
    b[1::3, :, :, 32:64] = a[::3, :, :, :32]
    slots = g.permutation(n + 1)[:n]
    start = g.integers(0, 40, n)
    first, count = g.integers(0, 31, n), g.integers(31, m + 1, n)
    first[:3], count[:3] = (0, 1, 30), (m, 31, 0)
    late = np.maximum(count - first, 0)
    # rows first.. in one call, rows 0..first in another: blocks shared by two calls keep both
    ka, vb = a.clone(), b.clone()
    for i in range(n):
        ka[i, :late[i]], vb[i, :late[i]] = a[i, first[i]:first[i] + late[i]], b[i, first[i]:first[i] + late[i]]
    c.append(ka, vb, i32(slots.tolist()), i32((start + first).tolist()), i32(late.tolist()))
    c.append(a, b, i32(slots.tolist()), i32(start.tolist()), i32(np.minimum(first, count).tolist()))
    fine(c)
    for typ in TYPES.values():
        rk, rv = c.read(i32(slots.tolist()), i32(start.tolist()), m, i32(count.tolist()), dtype=typ)
        for got, x in ((rk, a), (rv, b)):
            want, got = ref.values(host(x)), host(got)
            for i in range(n):
                np.testing.assert_array_equal(got[i, :count[i]], torch.from_numpy(want[i, :count[i]]).to(typ).double().numpy())
                assert not got[i, count[i]:].any()
    zeros = [0] * n
    before = [host(t) for t in c.read(i32(slots.tolist()), i32(zeros), cap, dtype=torch.float32)]
    for i in range(n):                                  # rows that no call named are as they were
        for x in before:
            assert not x[i, :start[i]].any() and not x[i, start[i] + count[i]:].any()
    bad = a.float()
    bad[2::5, ::7, :, 9], bad[3::5, ::5, :, d - 1] = float("nan"), float("-inf")
    if dtype != "f16":                                  # (the largest number is not one of fp16's)
        c.append(bad.to(a.dtype), bad.to(a.dtype), i32(slots.tolist()), i32(start.tolist()))
        rk, rv = c.read(i32(slots.tolist()), i32(start.tolist()), m, dtype=torch.float32)
        want = ref.values(host(bad.to(a.dtype)))
        np.testing.assert_array_equal(host(rk), want)
        np.testing.assert_array_equal(host(rv), want)
        from accelerator_decode_gb300 import g4
        assert c.device_error() == (g4.G4_ERR_DEVICE_CHECK, g4.G4_DEV_BAD_VALUE)
    if page:
        c._table[int(slots[0]), 0] = -1
        rk, rv = c.read(i32(slots.tolist()), i32(zeros), cap)
        assert not host(rk[0, :page]).any() and not host(rv[0, :page]).any()
        from accelerator_decode_gb300 import g4
        assert c.device_error() == (g4.G4_ERR_DEVICE_CHECK, g4.G4_DEV_BAD_POSITION)


def test_append_borders(rt):
    """Rounding ties, numbers one step beside a border, zero groups, the smallest and largest scales."""
    d, m = 128, 64
    g = np.random.default_rng(5)
    x = np.zeros((1, m, 1, d), np.float32)
    for r in range(m):
        for grp in range(d // 32):
            s = np.float32(ref.bf16_round(np.exp(g.uniform(-80, 80))))
            if r % 8 == 7:
                s = np.float32(2.0 ** g.integers(-133, -126))        # subnormal scales
            c = g.integers(-7, 7, 32) + 0.5
            v = (c * np.float64(s)).astype(np.float32)
            up = g.integers(-1, 2, 32)
            v = np.where(up > 0, np.nextafter(v, np.float32(np.inf)), np.where(up < 0, np.nextafter(v, np.float32(-np.inf)), v))
            v[0] = 7 * s
            x[0, r, 0, grp * 32:(grp + 1) * 32] = v
    x[0, 3] = 0
    x[0, 4, 0, 32:64] = 0
    x[0, 5, 0, :32] = np.float32(3.4e38)
    x[0, 5, 0, 32:64] = np.float32(1e-45)
    c = make(rt, 1, m, 1, 1, d)
    k = torch.from_numpy(x).cuda()
    c.append(k, -k, i32([0]), i32([0]))
    rk, rv = c.read(i32([0]), i32([0]), m, dtype=torch.float32)
    want = ref.values(x)
    np.testing.assert_array_equal(host(rk), want)
    np.testing.assert_array_equal(host(rv), -want)
    assert np.isfinite(host(rk)).all()
    fine(c)


def test_read_beyond_a_types_range(rt):
    """fp16 results hold infinities where a row's value is too large for them; the row keeps it."""
    x = torch.zeros(1, 2, 1, 64, device="cuda")
    x[0, 0, 0, 0], x[0, 0, 0, 40], x[0, 1, 0, 5] = 7e6, -7e5, 3.0
    c = make(rt, 1, 4, 1, 1, 64)
    c.append(x, -x, i32([0]), i32([0]))
    want = torch.from_numpy(ref.values(host(x)))
    for typ in TYPES.values():
        rk, rv = c.read(i32([0]), i32([0]), 2, dtype=typ)
        np.testing.assert_array_equal(host(rk), want.to(typ).double().numpy())
        np.testing.assert_array_equal(host(rv), (-want).to(typ).double().numpy())
    fine(c)


def test_append_not_finite(rt):
    """NaN is stored as 0, an infinity as the largest number; both are reported, neighbours are fine."""
    d = 64
    x = rows((1, 4, 1, d), "f32", 6)
    x[0, 1, 0, 3], x[0, 1, 0, 40], x[0, 2, 0, 0] = float("nan"), float("inf"), float("-inf")
    c = make(rt, 1, 8, 1, 1, d)
    c.append(x, x, i32([0]), i32([0]))
    rk, rv = c.read(i32([0]), i32([0]), 4, dtype=torch.float32)
    want = ref.values(host(x))
    np.testing.assert_array_equal(host(rk), want)
    np.testing.assert_array_equal(host(rv), want)
    from accelerator_decode_gb300 import g4
    assert c.device_error() == (g4.G4_ERR_DEVICE_CHECK, g4.G4_DEV_BAD_VALUE)
    fine(c)


# ------------------------------------------------------------------------- attention
def attend_bound(q, k, v, scale, dtype, want):
    """How far an element may be off.  A score is a sum of d products; each operand part beyond
    the kept bits and each of the d + 8 fp32 roundings costs at most 2^-23 of sum|q k| (the tensor
    core truncates where IEEE would round).  A weight p = exp(s - max) / sum then is off by at most
    the factor 1 + 2 ds + (the exponential's and the sum's (T + 8) 2^-23); a weight's kept bits
    (16 for outputs of 16 bits, 24 for fp32) cost another 2^-16 / 2^-23.  The output's rounding is
    eps / 2 of its value."""
    t, d = k.shape[0], k.shape[-1]
    qk = np.abs(q).reshape(-1, d).sum(1).max() * np.abs(k).max() if k.size else 0.0
    ds = scale * qk * (d + 8) * 2.0 ** -23
    dp = 2 * ds + (t + 8) * 2.0 ** -23 + (2.0 ** -23 if dtype == "f32" else 2.0 ** -16)
    vmax = np.abs(v).max() if v.size else 0.0
    eps = torch.finfo(TYPES[dtype]).eps / 2
    tiny = torch.finfo(TYPES[dtype]).smallest_normal * eps * 2
    return dp * vmax * (1 + eps) + eps * np.abs(want) + tiny


def check_attend(rt, d, kvh, group, lens, q_len, dtype, page=0, window=0, track=False, q_lens=None, scale=0.0, seed=0):
    n, heads, cap = len(lens), kvh * group, max(max(lens), 1) + 7
    c = make(rt, n + 1, cap, heads, kvh, d, page, max_q_len=q_len, track=track, seed=seed)
    slots = [(3 * i + 1) % (n + 1) for i in range(n)] if (n + 1) % 3 else list(range(n, 0, -1))
    k, v = rows((n, cap, kvh, d), dtype, seed + 10), rows((n, cap, kvh, d), dtype, seed + 11)
    k *= 0.5
    # rows behind a sequence's end hold large numbers that nothing may see
    c.append(k * 100, v * 100, i32(slots), i32([0] * n))
    finite = bool((k * 100).isfinite().all() and (v * 100).isfinite().all())   # fp16 may overflow here
    assert c.device_error()[1] == (0 if finite else 16)
    c.append(k, v, i32(slots), i32([0] * n), i32(lens))
    q = rows((n, q_len, heads, d), dtype, seed + 12)
    w0 = None
    if track:
        w0 = torch.rand(n, kvh, cap, generator=torch.Generator().manual_seed(seed)).cuda()
        c.append(k, v, i32(slots), i32([0] * n), i32(lens), weights=w0)
    out = torch.full((n, q_len, heads, d), 7.0, dtype=TYPES[dtype], device="cuda")
    got = c.attend(q, i32(slots), i32(lens), None if q_lens is None else i32(q_lens), scale=scale, window=window,
                   accumulate=track, out=out)
    assert got is out
    again = c.attend(q, i32(slots), i32(lens), None if q_lens is None else i32(q_lens), scale=scale, window=window)
    sc = scale or 1 / np.sqrt(d)
    for i in range(n):
        m = q_len if q_lens is None else q_lens[i]
        kk, vv = ref.values(host(k[i, :lens[i]])), ref.values(host(v[i, :lens[i]]))
        qq = host(q[i, :m])
        want, gain = ref.attend(qq, kk, vv, group, sc, window)
        bound = attend_bound(qq, kk, vv, sc, dtype, want)
        err = np.abs(host(out[i, :m]) - want)
        assert (err <= bound).all(), (i, float((err - bound).max()), float(err.max()))
        assert (host(out[i, m:]) == 7.0).all()
        assert torch.equal(again[i, :m], out[i, :m])
        if track:
            _, w = c.account(i32([slots[i]]), i32([0]), cap)
            wi = host(w[0, :, :lens[i]])
            w_want = host(w0[i, :, :lens[i]]) + gain
            qk = np.abs(qq).reshape(-1, d).sum(1).max() * np.abs(kk).max() if kk.size and qq.size else 0.0
            rel = 2 * sc * qk * (d + 8) * 2.0 ** -23 + (lens[i] + m * group + 16) * 2.0 ** -23
            assert (np.abs(wi - w_want) <= rel * (gain + 1e-30) + 2.0 ** -23 * np.abs(w_want)).all()
    fine(c)


LENS = [1, 15, 16, 17, 63, 64, 65, 130]


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("page", [0, 16, 128])
def test_decode(rt, d, dtype, page):
    check_attend(rt, d, 1, 8, [0] + LENS + [700], 1, dtype, page, seed=d)


@pytest.mark.parametrize("kvh,group", [(2, 1), (3, 2), (2, 5), (1, 16), (4, 7), (1, 40)])
def test_decode_head_groups(rt, kvh, group):
    check_attend(rt, 128, kvh, group, LENS, 1, "bf16", 32, seed=group)


@pytest.mark.parametrize("window", [1, 16, 63, 64, 512])
@pytest.mark.parametrize("q_len", [1, 5])
def test_window(rt, window, q_len):
    check_attend(rt, 64, 2, 4, [5, 16, 17, 64, 65, 600], q_len, "f32", 16, window=window, seed=window)


@pytest.mark.parametrize("d,q_len,group", [(64, 7, 3), (128, 64, 4), (256, 33, 8), (512, 9, 8), (256, 2, 4), (256, 64, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_block(rt, d, q_len, group, dtype):
    """Several query tokens per sequence, causal; more tokens than rows leaves empty ones."""
    lens = [q_len, q_len + 1, 200, 3, 513, 0]
    check_attend(rt, d, 2, group, lens, q_len, dtype, 64, q_lens=[q_len, max(1, q_len // 2), q_len, q_len, 1, q_len],
                 seed=d + q_len)


@pytest.mark.parametrize("q_len,group,kvh", [(1, 8, 1), (1, 3, 4), (1, 20, 2), (6, 4, 2), (64, 8, 1)])
@pytest.mark.parametrize("dtype,d,page", [("bf16", 256, 128), ("f32", 64, 0), ("f16", 512, 16)])
def test_account(rt, q_len, group, kvh, dtype, d, page):
    check_attend(rt, d, kvh, group, [0, q_len, 64, 65, 700], q_len, dtype, page, track=True, seed=q_len + group)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len,group,kvh,page", [(5, 7, 1, 0), (33, 1, 2, 16), (64, 8, 1, 64), (17, 16, 3, 128)])
@pytest.mark.parametrize("track", [False, True])
def test_token_blocks(rt, d, q_len, group, kvh, page, track):
    """More than 32 query rows per KV head: ragged tokens, prompts shorter than a tile, rows that no
    tile reaches, items shared by many CTAs."""
    lens = [q_len, 0, 64, 65, 700, 1, 2051]
    q_lens = [q_len, q_len, max(1, q_len - 3), 1, q_len, q_len, q_len // 2]
    check_attend(rt, d, kvh, group, lens, q_len, "bf16", page, q_lens=q_lens, track=track, seed=d + q_len)


@pytest.mark.parametrize("d,kvh", [(256, 2), (128, 4), (64, 2)])
@pytest.mark.parametrize("track", [False, True])
def test_token_blocks_many_tiles(rt, d, kvh, track):
    """A batch whose CTAs each take many tiles in a row, several items and odd numbers of them."""
    n, q_len, group, cap = 40, 36, 4, 1500
    lens = [36 + (i * 977) % 1465 for i in range(n)]
    c = make(rt, n, cap, kvh * group, kvh, d, 64, track=track)
    k, v = rows((n, cap, kvh, d), "bf16", 1), rows((n, cap, kvh, d), "bf16", 2)
    slots = list(range(n))
    c.append(k, v, i32(slots), i32([0] * n), i32(lens))
    q = rows((n, q_len, kvh * group, d), "bf16", 3)
    out = c.attend(q, i32(slots), i32(lens), accumulate=track)
    fine(c)
    for i in range(n):
        kk, vv = (torch.from_numpy(ref.values(host(x[i, :lens[i]]))).cuda() for x in (k, v))
        qq = q[i].double().reshape(q_len, kvh, group, d)
        s = torch.einsum("mkgd,tkd->kgmt", qq, kk) / np.sqrt(d)
        j, last = torch.arange(lens[i], device="cuda"), lens[i] - q_len + torch.arange(q_len, device="cuda")
        p = torch.softmax(s.masked_fill(j > last[:, None], -np.inf), -1)
        want = torch.einsum("kgmt,tkd->mkgd", p, vv).reshape(q_len, kvh * group, d)
        bound = attend_bound(host(q[i]), host(kk), host(vv), 1 / np.sqrt(d), "bf16", host(want))
        assert (np.abs(host(out[i]) - host(want)) <= bound).all()
        # far inside that worst case: an rms error is the output's rounding (2^-9 / sqrt 3 of the value) and little else
        assert (out[i].double() - want).norm() <= 2.0 ** -8 * want.norm()
        if track:
            _, w = c.account(i32([i]), i32([0]), lens[i])
            gain = p.sum((1, 2))
            assert (w[0].double() - gain).norm() <= 2e-5 * gain.norm()


@pytest.mark.parametrize("window", [1, 63, 64, 300])
def test_token_block_window(rt, window):
    check_attend(rt, 128, 2, 8, [9, 64, 65, 900, 40], 9, "bf16", 32, window=window, seed=window)


def test_long_context(rt):
    check_attend(rt, 256, 1, 8, [30011, 5], 1, "bf16", 128, track=True, seed=3)
    check_attend(rt, 64, 1, 2, [40007, 39000, 1], 1, "f32", 0, scale=0.03, seed=4)


def test_strided_query_and_output(rt):
    """Heads outside tokens, a broadcast query, an output whose base is not 16-byte aligned."""
    n, kvh, group, d, t, m = 2, 2, 2, 64, 50, 3
    c = make(rt, n, 64, kvh * group, kvh, d)
    k, v = rows((n, t, kvh, d), "bf16", 1), rows((n, t, kvh, d), "bf16", 2)
    c.append(k, v, i32([0, 1]), i32([0, 0]))
    q = rows((n, kvh * group, m, d), "bf16", 3)
    want = c.attend(q.transpose(1, 2).contiguous(), i32([0, 1]), i32([t, t]))
    buf = torch.zeros(n, kvh * group, m, d + 5, dtype=torch.bfloat16, device="cuda")
    out = buf.transpose(1, 2)[..., 1:1 + d]
    c.attend(q.transpose(1, 2), i32([0, 1]), i32([t, t]), out=out)
    assert torch.equal(out, want)
    assert not buf[..., 0].any() and not buf[..., 1 + d:].any()
    one = q[:1, :, :1].transpose(1, 2)
    a = c.attend(one.expand(n, m, kvh * group, d), i32([0, 1]), i32([t, t]))
    b = c.attend(one.expand(n, m, kvh * group, d).contiguous(), i32([0, 1]), i32([t, t]))
    assert torch.equal(a, b)
    fine(c)


def test_packed_projection_and_extreme_arguments(rt):
    """Queries, keys, values and the output as slices of one packed tensor; a window past every row;
    scales at both ends; one sequence more than the spans of a block kernel hold."""
    n, kvh, group, d, t = 2, 2, 3, 128, 70
    heads = kvh * group
    pack = rows((n, t, heads + 2 * kvh + heads, d), "bf16", 1)
    q, k, v, out = pack[:, :, :heads], pack[:, :, heads:heads + kvh], pack[:, :, heads + kvh:heads + 2 * kvh], pack[:, :, heads + 2 * kvh:]
    c = make(rt, n, 128, heads, kvh, d, 16)
    c.append(k, v, i32([0, 1]), i32([0, 0]))
    lens, slots, m = i32([t, t]), i32([0, 1]), 9
    want = c.attend(q[:, -m:].contiguous(), slots, lens)
    before = pack[:, :, :heads + 2 * kvh].clone()
    c.attend(q[:, -m:], slots, lens, out=out[:, -m:])
    assert torch.equal(out[:, -m:], want) and torch.equal(pack[:, :, :heads + 2 * kvh], before)
    for w in (128, 1000, (1 << 31) - 1):
        assert torch.equal(c.attend(q[:, -m:], slots, lens, window=w), want)
    assert torch.equal(c.attend(q[:, -m:], slots, lens, window=127), want)
    for scale in (1e-38, 1e30):
        assert c.attend(q[:, -m:], slots, lens, scale=scale).isfinite().all() or scale > 1
    one = c.attend(q[:, -m:], slots, lens, scale=1e-38)              # equal weights: the mean of the seen rows
    vals = torch.from_numpy(ref.values(host(v[0])))
    np.testing.assert_allclose(host(one[0, -1, 0]), vals[:, 0].mean(0), rtol=2.0 ** -7, atol=2.0 ** -8)
    many = make(rt, 400, 20, 40, 1, 64)
    kk, qq = rows((400, 3, 1, 64), "bf16", 2), rows((400, 1, 40, 64), "bf16", 3)
    order = i32(list(range(400)))
    many.append(kk, kk, order, i32([0] * 400))
    whole = many.attend(qq, order, i32([3] * 400))
    part = many.attend(qq[:100], order[:100], i32([3] * 100))
    assert (whole[:100].float() - part.float()).abs().max() <= 2.0 ** -7 * part.float().abs().max()
    fine(c)
    fine(many)


@pytest.mark.parametrize("m,dtype", [(2, "f32"), (2, "bf16"), (6, "bf16")])
def test_not_finite_query_stays_in_its_row(rt, m, dtype):
    d, t = 128, 100
    c = make(rt, 1, 128, 8, 1, d)
    c.append(rows((1, t, 1, d), "f32", 1), rows((1, t, 1, d), "f32", 2), i32([0]), i32([0]))
    q = rows((1, m, 8, d), dtype, 3)
    clean = c.attend(q, i32([0]), i32([t]))
    q[0, 1, 3, 5] = float("nan")
    q[0, 0, 6, 0] = float("inf")
    out = c.attend(q, i32([0]), i32([t]))
    bad = torch.zeros(m, 8, dtype=torch.bool)
    bad[1, 3] = bad[0, 6] = True
    assert out[0][bad.cuda()].isnan().all()
    assert torch.equal(out[0][~bad.cuda()], clean[0][~bad.cuda()])


# -------------------------------------------------------------------------- eviction
def evict_check(rt, lens, budget, recent, kvh=2, d=64, page=16, ties=False, special=False, seed=0):
    n, cap = len(lens), max(max(lens), budget, 1)
    c = make(rt, n, cap, kvh, kvh, d, page, track=True, seed=seed)
    g = np.random.default_rng(seed)
    k, v = rows((n, cap, kvh, d), "f32", seed + 1), rows((n, cap, kvh, d), "f32", seed + 2)
    w = (g.integers(0, 4, (n, kvh, cap)) if ties else g.exponential(1, (n, kvh, cap))).astype(np.float32)
    if special:
        w[..., ::3] = np.nan
        w[..., 1::5] = -np.inf
        w[..., 2::7] = np.inf
        w[..., 3::7] = -0.0
        w[..., 4::11] = 0.0
        w[..., 5::13] = -1.5
    pos = np.stack([np.stack([g.permutation(3 * cap)[:cap] for _ in range(kvh)]) for _ in range(n)]).astype(np.int32)
    slots = i32(list(range(n))[::-1])
    c.append(k, v, slots, i32([0] * n), i32(lens), positions=torch.from_numpy(pos).cuda(), weights=torch.from_numpy(w).cuda())
    new = c.evict(slots, i32(lens), budget, recent)
    assert new.tolist() == [min(x, budget) for x in lens]
    gp, gw = c.account(slots, i32([0] * n), cap)
    gk, gv = c.read(slots, i32([0] * n), cap, dtype=torch.float32)
    vk, vv = ref.values(host(k)), ref.values(host(v))
    for i, ln in enumerate(lens):
        for h in range(kvh):
            src = ref.evict_source(pos[i, h, :ln], w[i, h, :ln], budget, recent)
            m = len(src)
            np.testing.assert_array_equal(gp[i, h, :m].cpu().numpy(), pos[i, h, src])
            np.testing.assert_array_equal(gw[i, h, :m].cpu().numpy(), w[i, h, src])
            np.testing.assert_array_equal(host(gk[i, :m, h]), vk[i, src, h])
            np.testing.assert_array_equal(host(gv[i, :m, h]), vv[i, src, h])
            # rows at and beyond the budget are left as they were
            np.testing.assert_array_equal(host(gk[i, budget:ln, h]), vk[i, budget:ln, h])
    fine(c)


@pytest.mark.parametrize("lens,budget,recent", [
    ([0, 1, 5, 6, 7, 33], 6, 2), ([40, 41, 17], 16, 0), ([100, 99], 33, 33), ([300, 1000, 2049], 257, 31),
    ([2], 1, 1), ([5000], 1024, 100)])
@pytest.mark.parametrize("ties,special", [(False, False), (True, False), (False, True)])
def test_evict(rt, lens, budget, recent, ties, special):
    evict_check(rt, lens, budget, recent, ties=ties, special=special, seed=budget)


def test_evict_more_rows_than_shared_memory_holds(rt):
    """60,000 rows of one head: the ranks are read anew in each pass."""
    evict_check(rt, [60000, 58000], 30001, 700, kvh=1, d=64, page=128, seed=1)
    evict_check(rt, [60000], 100, 3, kvh=1, d=64, page=0, ties=True, seed=2)


@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_evict_head_dims(rt, d):
    evict_check(rt, [70, 64], 33, 5, kvh=3, d=d, page=0, seed=d)


# ------------------------------------------------------------------ used together
@pytest.mark.parametrize("page,dtype", [(0, "f32"), (32, "bf16")])
def test_bounded_session(rt, page, dtype):
    """Prompt blocks and single tokens through append, attend with account, and evict, with the
    rows held on the host beside them; whole numbers are compared at every step."""
    n, kvh, group, d, budget, recent = 3, 2, 3, 64, 40, 9
    c = make(rt, n, 128, kvh * group, kvh, d, page, max_q_len=32, track=True)
    slots = [2, 0, 1]
    held = [dict(k=np.zeros((kvh, 0, d)), v=np.zeros((kvh, 0, d)), p=np.zeros((kvh, 0), np.int32)) for _ in range(n)]
    lens, seen = [0] * n, 0
    for step, m in enumerate([32, 32, 1, 1, 7, 1, 1]):
        k, v = rows((n, m, kvh, d), dtype, 100 + step), rows((n, m, kvh, d), dtype, 200 + step)
        q = rows((n, m, kvh * group, d), dtype, 300 + step)
        pos = torch.arange(seen, seen + m, dtype=torch.int32, device="cuda").expand(n, kvh, m).contiguous()
        c.append(k, v, i32(slots), i32(lens), positions=pos)
        lens = [x + m for x in lens]
        out = c.attend(q, i32(slots), i32(lens), accumulate=True)
        for i in range(n):
            hd = held[i]
            hd["k"] = np.concatenate([hd["k"], ref.values(host(k[i])).transpose(1, 0, 2)], 1)
            hd["v"] = np.concatenate([hd["v"], ref.values(host(v[i])).transpose(1, 0, 2)], 1)
            hd["p"] = np.concatenate([hd["p"], np.tile(np.arange(seen, seen + m, dtype=np.int32), (kvh, 1))], 1)
            kk, vv = hd["k"].transpose(1, 0, 2), hd["v"].transpose(1, 0, 2)
            want, _ = ref.attend(host(q[i]), kk, vv, group, 1 / np.sqrt(d))
            bound = attend_bound(host(q[i]), kk, vv, 1 / np.sqrt(d), dtype, want)
            assert (np.abs(host(out[i]) - want) <= bound).all()
        seen += m
        pos_now, w = c.account(i32(slots), i32([0] * n), lens[0])
        for i in range(n):
            np.testing.assert_array_equal(pos_now[i].cpu().numpy(), held[i]["p"])
        new = c.evict(i32(slots), i32(lens), budget, recent)
        for i in range(n):
            hd, wi = held[i], w[i].cpu().numpy()
            src = [ref.evict_source(hd["p"][h], wi[h], budget, recent) for h in range(kvh)]
            for key in ("k", "v", "p"):
                hd[key] = np.stack([hd[key][h][src[h]] for h in range(kvh)])
        lens = new.tolist()
        assert lens == [min(seen, budget)] * n or lens == [len(held[0]["p"][0])] * n
        pos_now, _ = c.account(i32(slots), i32([0] * n), lens[0])
        for i in range(n):
            np.testing.assert_array_equal(pos_now[i].cpu().numpy(), held[i]["p"])
            assert (held[i]["p"].max(1) == seen - 1).all()
    fine(c)


# ------------------------------------------------------------- refusals and errors
def test_refusals(rt):
    from accelerator_decode_gb300 import g4
    d = 64
    c = make(rt, 4, 32, 4, 2, d, max_q_len=4)
    t = make(rt, 4, 32, 4, 2, d, max_q_len=4, track=True)
    k, q = rows((2, 3, 2, d), "f32", 1), rows((2, 2, 4, d), "f32", 2)
    s, z, l = i32([0, 1]), i32([0, 0]), i32([3, 3])
    pos, w = torch.zeros(2, 2, 3, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, 3, device="cuda")

    def refused(status, fn, *a, **kw):
        with pytest.raises(g4.G4Error) as e:
            fn(*a, **kw)
        assert e.value.status == status

    bad, uns = g4.G4_ERR_INVALID_ARG, g4.G4_ERR_UNSUPPORTED
    refused(uns, c.append, k, k, s, z, positions=pos)
    refused(uns, c.append, k, k, s, z, weights=w)
    refused(uns, c.account, s, z, 3)
    refused(uns, c.evict, s, l, 2)
    refused(uns, c.attend, q, s, l, accumulate=True)
    refused(uns, t.attend, q, s, l, window=4)
    refused(bad, c.attend, q, s, l, window=-1)
    for scale in (float("inf"), float("nan"), -0.5):
        refused(bad, c.attend, q, s, l, scale=scale)
    refused(bad, c.attend, q, s, l, out=torch.empty(2, 2, 4, d, dtype=torch.bfloat16, device="cuda"))
    refused(bad, c.attend, q, s, l, out=torch.empty(2, 2, 1, d, device="cuda").expand(2, 2, 4, d))
    refused(bad, c.attend, rows((2, 5, 4, d), "f32", 2), s, l)
    refused(bad, c.attend, q, s, l, out=q)
    refused(bad, c.read, s, z, 33)
    refused(bad, c.read, s, z, 0)
    refused(bad, t.evict, s, l, 0)
    refused(bad, t.evict, s, l, 33)
    refused(bad, t.evict, s, l, 4, 5)
    refused(bad, t.evict, s, l, 4, -1)
    for args in ((k[..., :32], k, s, z), (k, k[:, :2], s, z), (k, k, s, z[:1]), (k.cpu(), k, s, z), (k, k, s.long(), z),
                 (k.double(), k, s, z), (k.transpose(2, 3).contiguous().transpose(2, 3), k, s, z)):
        with pytest.raises((ValueError, TypeError)):
            c.append(*args)
    five = i32([0, 1, 2, 3, 0])
    refused(bad, c.read, five, five, 3)
    assert c.device_bytes() > 0
    fine(c)
    fine(t)


def test_device_errors_skip_the_sequence(rt):
    """Bad slots, rows and counts cost their own sequence only, and are reported."""
    from accelerator_decode_gb300 import g4
    d, m = 64, 4
    c = make(rt, 6, 20, 2, 1, d, track=True)
    k = rows((6, m, 1, d), "f32", 1)
    c.append(k, k, i32([0, 6, -1, 3, 4, 0]), i32([0, 0, 0, 17, -1, 8]))
    assert c.device_error() == (g4.G4_ERR_DEVICE_CHECK, g4.G4_DEV_BAD_SLOT | g4.G4_DEV_BAD_POSITION)
    rk, _ = c.read(i32([0, 1, 2, 3, 4, 5]), i32([0] * 6), 20, dtype=torch.float32)
    np.testing.assert_array_equal(host(rk[0, :m]), ref.values(host(k[0])))
    assert not host(rk[0, m:]).any() and not host(rk[1:]).any()
    fine(c)
    c.append(k[:2], k[:2], i32([1, 2]), i32([0, 0]), i32([5, -1]))
    assert c.device_error()[1] == g4.G4_DEV_BAD_POSITION
    q = rows((4, 2, 2, d), "f32", 2)
    good = c.attend(q[:1], i32([0]), i32([4]))
    for slots, lens in (([0, 7, 0, 1], [4, 4, 21, -1]), ([0, -5, 2, 3], [4, 4, 1 << 30, -(1 << 31)])):
        out = c.attend(q, i32(slots), i32(lens))
        assert torch.equal(out[:1], good) and not out[1:].any()
        assert c.device_error()[1] == g4.G4_DEV_BAD_SLOT | g4.G4_DEV_BAD_POSITION
    out = c.attend(q, i32([0] * 4), i32([4] * 4))                # naming a slot twice is fine for reading
    assert torch.equal(out[3], c.attend(q[3:], i32([0]), i32([4]))[0])
    fine(c)
    out = c.attend(q[:2], i32([0, 0]), i32([4, 4]), accumulate=True)
    assert torch.equal(out[:1], good) and not out[1:].any()
    assert c.device_error()[1] == g4.G4_DEV_BAD_SLOT
    _, w = c.account(i32([0]), i32([0]), 4)
    assert abs(float(w.sum()) - 4) < 1e-5                        # two tokens, two heads, once
    out = c.attend(q[:2], i32([0, 0]), i32([4, 4]), q_lens=i32([3, -1]))
    assert not out.any() and c.device_error()[1] == g4.G4_DEV_BAD_POSITION
    new = c.evict(i32([0, 0, 9]), i32([4, 4, 4]), 2)
    assert new.tolist() == [2, 4, 4] and c.device_error()[1] == g4.G4_DEV_BAD_SLOT
    pos, w = c.account(i32([0, 11]), i32([19, 0]), 2)
    assert c.device_error()[1] == g4.G4_DEV_BAD_SLOT | g4.G4_DEV_BAD_POSITION


@pytest.mark.parametrize("m,group", [(1, 2), (5, 8)])
def test_missing_pages(rt, m, group):
    """Rows on missing pages are not written, read or seen; the others are."""
    from accelerator_decode_gb300 import g4
    d, t = 64, 64
    heads, dtype = group, "f32" if m == 1 else "bf16"
    table = torch.tensor([[1, -1, 4, 0], [2, 3, 99, 5]], dtype=torch.int32, device="cuda")
    c = make(rt, 2, t, heads, 1, d, 16, page_table=table, n_pages=6, track=True)
    k, v = rows((2, t, 1, d), "f32", 1), rows((2, t, 1, d), "f32", 2)
    c.append(k, v, i32([0, 1]), i32([0, 0]))
    assert c.device_error()[1] == g4.G4_DEV_BAD_POSITION
    q = rows((2, m, heads, d), dtype, 3)
    out = c.attend(q, i32([0, 1]), i32([t, t]), accumulate=True)
    assert c.device_error()[1] == g4.G4_DEV_BAD_POSITION
    for i, gone in enumerate([(16, 32), (32, 48)]):
        keep = np.r_[0:gone[0], gone[1]:t]
        kk, vv = ref.values(host(k[i]))[keep], ref.values(host(v[i]))[keep]
        want, gain = ref.attend(host(q[i]), kk, vv, group, 1 / np.sqrt(d))
        assert (np.abs(host(out[i]) - want) <= attend_bound(host(q[i]), kk, vv, 1 / np.sqrt(d), dtype, want)).all()
        _, w = c.account(i32([i]), i32([0]), t)
        assert np.abs(host(w[0, 0])[keep] - gain[0]).max() < 1e-4 * m * group and not host(w[0, 0])[gone[0]:gone[1]].any()
    c.device_error()
    rk, _ = c.read(i32([0, 1]), i32([0, 0]), t, i32([t, t]), dtype=torch.float32)
    assert c.device_error()[1] == g4.G4_DEV_BAD_POSITION
    np.testing.assert_array_equal(host(rk[0, :16]), ref.values(host(k[0, :16])))
    assert not host(rk[0, 16:32]).any()
    new = c.evict(i32([0, 1]), i32([t, 32]), 10)                 # a slot with a missing page is not cut
    assert new.tolist() == [t, 10] and c.device_error()[1] == g4.G4_DEV_BAD_POSITION
    fine(c)


# --------------------------------------------------------------- streams and graphs
def test_other_stream_and_graph(rt):
    """The calls on a side stream, and captured once and replayed on new inputs in place."""
    n, d, t = 2, 128, 90
    c = make(rt, n, 128, 8, 1, d, 16, track=True)
    other = make(rt, n, 128, 8, 1, d, 16, track=True)
    k, v = rows((n, t, 1, d), "bf16", 1), rows((n, t, 1, d), "bf16", 2)
    for x in (c, other):
        x.append(k, v, i32([0, 1]), i32([0, 0]))
    slots, start, lens = i32([0, 1]), i32([t, t]), i32([t + 1, t + 1])
    k1, v1, q = (rows((n, 1, h, d), "bf16", s) for h, s in ((1, 3), (1, 4), (8, 5)))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.empty_like(q)

    def step(x, o, stream=None):
        x.append(k1, v1, slots, start, stream=stream)
        x.attend(q, slots, lens, accumulate=True, out=o, stream=stream)
        return x.evict(slots, lens, t, 8, stream=stream)

    want = torch.empty_like(q)
    step(other, want)
    torch.cuda.synchronize()
    step(c, out, side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new = step(c, out)
    for seed in (7, 8):
        for dst, s in ((k1, seed), (v1, seed + 10), (q, seed + 20)):
            dst.copy_(rows(tuple(dst.shape), "bf16", s))
        graph.replay()
        step(other, want)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and new.tolist() == [t, t]
        for x, y in zip(c.account(slots, i32([0, 0]), t), other.account(slots, i32([0, 0]), t)):
            assert torch.equal(x, y)
        for x, y in zip(c.read(slots, i32([0, 0]), t), other.read(slots, i32([0, 0]), t)):
            assert torch.equal(x, y)
    fine(c)


def test_split_layouts_agree_with_one_sequence_at_a_time(rt):
    """A ragged batch gives the bits that each sequence's own bound allows, and every slot its own."""
    n, d, kvh = 9, 256, 2
    lens = [1, 2000, 3, 64, 777, 0, 128, 129, 1500]
    c = make(rt, n, 2048, 8, kvh, d, 128)
    k, v = rows((n, 2048, kvh, d), "bf16", 1), rows((n, 2048, kvh, d), "bf16", 2)
    c.append(k, v, i32(list(range(n))), i32([0] * n), i32(lens))
    q = rows((n, 1, 8, d), "bf16", 3)
    whole = c.attend(q, i32(list(range(n))), i32(lens))
    for i, ln in enumerate(lens):
        one = c.attend(q[i:i + 1], i32([i]), i32([ln]))
        kk, vv = ref.values(host(k[i, :ln])), ref.values(host(v[i, :ln]))
        bound = attend_bound(host(q[i]), kk, vv, 1 / 16, "bf16", host(one[0]))
        assert (np.abs(host(whole[i]) - host(one[0])) <= 2 * bound).all()
    fine(c)
