"""Attention over 16-bit keys and values on the GPU against 64 bits (kv4_accuracy.attend).

Errors are taken per output row as |error| / |row| (kv4_accuracy explains why rows are sums of many
independent errors).  With u = eps / 2 of the type, an output row is off by
* its own rounding: 0.65 u in the root mean square, at most u (`few`);
* its weights' rounding into the products: each weight is off by at most u of itself, independently
  of the others, which moves the row as its own rounding does: 0.65 u, or for a row of few keys at most
  u sum p |v| / |sum p v|, which for the random values here (angles near a right one) is below 1.5 u;
  fp16 weights below 2^-14 are off by up to 2^-25 each at the most, and n of them by 2^-25 sqrt(n) of a value;
* scores: d / 16 steps, each off by at most 2^-23 of numbers below 4 after the scale; twice that;
* the exponential's 2^-22 and 2^-23 for each of the (keys / 16 + 32) steps of the sums."""
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


def limit(dtype, d, keys):
    u = torch.finfo(TYPES[dtype]).eps / 2
    few = keys < 64
    small = 2.0 ** -25 * math.sqrt(keys) if dtype == "f16" else 0.0
    return (2.5 if few else 1.3) * u + 2 * d / 16 * 4 * 2.0 ** -23 + 2.0 ** -22 + (keys / 16 + 32) * 2.0 ** -23 + 4 * small


def right(out, want, dtype, keys):
    """Every row within its limit, whose keys' number `keys` gives (a list or one number)."""
    errors = acc.row_errors(out.cpu(), want.cpu())
    ks = keys if isinstance(keys, list) else [keys] * errors.shape[0]
    lim = torch.tensor([limit(dtype, out.shape[-1], k) for k in ks]).double()[:, None]
    bad = ~(errors <= lim)
    assert not bad.any(), (bad.nonzero()[:5].tolist(), errors[bad][:5].tolist(), lim.flatten()[:3].tolist())


def packed(lens, heads, kvh, d, dtype, seed, front=0, rest=0):
    """q, k, v of packed sequences with `front` and `rest` rows around them that hold NaN."""
    n = sum(lens)
    q, k, v = acc.inputs(1, n, kvh, heads // kvh, n, d, dtype, seed)
    pad = lambda x: torch.cat([torch.full((front, *x.shape[2:]), math.nan).to(x), x[0],
                               torch.full((rest, *x.shape[2:]), math.nan).to(x)]).cuda()
    offsets = [front]
    for m in lens:
        offsets.append(offsets[-1] + m)
    return pad(q), pad(k), pad(v), offsets


def check_prompt(out, q, k, v, offsets, dtype, window=0, scale=None):
    for a, b in zip(offsets, offsets[1:]):
        if a == b:
            continue
        want, _ = acc.attend(q[a:b], k[a:b], v[a:b], scale, window)
        keys = [min(i + 1, window or i + 1) for i in range(b - a)]
        right(out[a:b], want, dtype, keys)


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype,heads,kvh", [("bf16", 4, 1), ("f16", 6, 2), ("bf16", 3, 3), ("bf16", 10, 2)])
@pytest.mark.parametrize("lens,window", [([1], 0), ([5, 0, 1, 130], 0), ([128], 0), ([300, 129, 17], 0), ([300, 129, 17], 40),
                                         ([513], 128), ([270, 64], 1)])
def test_prompt(rt, d, dtype, heads, kvh, lens, window):
    """Lengths around a tile, empty sequences, odd groups, windows; NaN around the sequences."""
    front, rest = (3, 5) if len(lens) > 1 else (0, 0)
    q, k, v, offsets = packed(lens, heads, kvh, d, dtype, sum(lens) + d, front, rest)
    a = rt.Attention(heads, kvh, d, dtype=TYPES[dtype], max_seqs=len(lens))
    out = a.prompt(q, k, v, i32(offsets), window=window)
    assert a.device_error() == (0, 0)
    assert not out[:front].any() and not out[offsets[-1]:].any()
    check_prompt(out, q, k, v, offsets, dtype, window)
    again = a.prompt(q, k, v, i32(offsets), window=window)
    assert torch.equal(out, again)


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("heads,kvh", [(64, 1), (43, 1), (86, 2), (22, 1)])
def test_prompt_wide_groups(rt, d, heads, kvh):
    """Groups of up to 64 heads: blocks of two tokens, and of fewer than 128 rows."""
    lens = [3, 131, 0, 40]
    q, k, v, offsets = packed(lens, heads, kvh, d, "bf16", heads, 1, 2)
    a = rt.Attention(heads, kvh, d, max_seqs=4)
    check_prompt(a.prompt(q, k, v, i32(offsets)), q, k, v, offsets, "bf16")
    assert a.device_error() == (0, 0)


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("heads,kvh,t,window", [(8, 1, 1500, 0), (8, 2, 2050, 512), (2, 2, 3001, 0)])
def test_prompt_long(rt, d, heads, kvh, t, window):
    lens = [t, t // 3, 1, t // 2 + 7]
    q, k, v, offsets = packed(lens, heads, kvh, d, "bf16", t + d)
    a = rt.Attention(heads, kvh, d, max_seqs=4)
    out = a.prompt(q, k, v, i32(offsets), window=window)
    assert a.device_error() == (0, 0)
    check_prompt(out, q, k, v, offsets, "bf16", window)


def pool_of(rt, lens, shared, kvh, d, dtype, page, seed, spare=1):
    """A table whose slot i holds lens[i] rows, the first `shared` pages those of slot len(lens), and pools
    with random rows; also dense keys and values of every slot."""
    n = len(lens)
    pages = shared + sum(max(0, -(-m // page) - shared) for m in lens) + spare
    most = max([shared] + [-(-m // page) for m in lens]) + 1
    t = rt.PageTable(n + 1, pages, page, most)
    rows = []
    if shared:
        rows.append(t.extend(i32([n]), i32([shared * page]), shared * page)[0])
        full = [i for i in range(n) if lens[i] >= shared * page]
        t.share(i32(full), n, shared)
    g = torch.Generator().manual_seed(seed)
    pools = [torch.full((pages, kvh, page, d), math.nan).to(TYPES[dtype]).cuda() for _ in "kv"]
    base = shared * page
    _, k, v = acc.inputs(1, base + sum(max(0, m - base) for m in lens) + 1, kvh, 1, 1, d, dtype, seed)
    k, v = k[0].cuda(), v[0].cuda()
    if shared:
        t.store(k[:base], v[:base], rows[0], *pools)
    at, dense = base, []
    left = [max(0, m - base) if m >= base else 0 for m in lens]
    where = [[] for _ in lens]
    while any(left):                                     # grown in turns: scattered pages
        step = [min(x, int(torch.randint(1, 3 * page, (1,), generator=g))) for x in left]
        r, o, _ = t.extend(i32(list(range(n))), i32(step), sum(step))
        t.store(k[at:at + sum(step)], v[at:at + sum(step)], r, *pools)
        for i, c in enumerate(step):
            where[i] += range(at + sum(step[:i]), at + sum(step[:i + 1]))
            left[i] -= c
        at += sum(step)
    for i, m in enumerate(lens):
        idx = torch.tensor(list(range(base)) + where[i] if m >= base else [], dtype=torch.long, device="cuda")
        dense.append((k[idx], v[idx]))
    return t, pools, dense


def check_shared(rt, a, t, pools, dense, shared, heads, kvh, d, dtype, slots=None, seed=0):
    slots = list(range(len(dense))) if slots is None else slots
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(len(slots), heads, d, generator=g).to(TYPES[dtype]).cuda()
    out = a.shared(q, *pools, t, i32(slots), shared)
    assert a.device_error() == (0, 0) and t.device_error() == (0, 0)
    for i, s in enumerate(slots):
        k, v = dense[s]
        if len(k) == 0:
            assert not out[i].any()
            continue
        want, _ = acc.attend(q[i:i + 1], k, v)
        right(out[i:i + 1], want, dtype, len(k))
    return q, out


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype,heads,kvh,page", [("bf16", 8, 1, 128), ("f16", 6, 2, 16), ("bf16", 10, 2, 64), ("f16", 32, 2, 256)])
@pytest.mark.parametrize("shared,lens", [(0, [1, 16, 0, 333]), (1, [0, 1, 17, 300]), (5, [1, 64, 700, 2, 3, 130])])
def test_shared(rt, d, dtype, heads, kvh, page, shared, lens):
    """Rows behind the prefix from none on, empty slots, pages below and above a tile; NaN where no row is."""
    lens = [shared * page + m - 1 if shared else m for m in lens]
    if shared:
        lens[0] = 0
    t, pools, dense = pool_of(rt, lens, shared, kvh, d, dtype, page, d + page)
    a = rt.Attention(heads, kvh, d, dtype=TYPES[dtype], max_seqs=len(lens))
    q, out = check_shared(rt, a, t, pools, dense, shared, heads, kvh, d, dtype, seed=heads)
    assert torch.equal(out, a.shared(q, *pools, t, i32(list(range(len(lens)))), shared))


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype,heads,kvh,page,n,rows", [
    ("bf16", 8, 1, 128, 40, 1408), ("f16", 6, 2, 16, 47, 1520), ("bf16", 10, 2, 64, 33, 1344), ("f16", 64, 1, 32, 24, 2144),
    ("bf16", 32, 8, 256, 21, 1280)])
def test_shared_once(rt, d, dtype, heads, kvh, page, n, rows):
    """Prefixes and batches beyond the bytes that each sequence reads on its own: the shared rows attended to once,
    in several parts and blocks of query rows; odd groups, pages below and above a tile, tiles cut short, empty
    slots, sequences without rows of their own."""
    n, rows = (2 * n, rows) if kvh * d < 128 else (n, rows)
    assert 4 * n * rows * kvh * d > 20e6 and rows > 1024 and rows % page == 0
    lens = [0 if i % 11 == 5 else rows + (37 * i * i) % 200 if i % 7 else rows for i in range(n)]
    t, pools, dense = pool_of(rt, lens, rows // page, kvh, d, dtype, page, d + n)
    a = rt.Attention(heads, kvh, d, dtype=TYPES[dtype], max_seqs=n)
    slots = list(range(n))[::-1]
    q, out = check_shared(rt, a, t, pools, dense, rows // page, heads, kvh, d, dtype, slots=slots, seed=heads)
    assert torch.equal(out, a.shared(q, *pools, t, i32(slots), rows // page))


@pytest.mark.parametrize("d", [64, 256])
def test_shared_many(rt, d):
    """1,024 sequences, and one whose rows fill many parts; a slot named more than once."""
    lens = [16 + (7 * i) % 23 for i in range(1023)]
    t, pools, dense = pool_of(rt, lens, 1, 1, d, "bf16", 16, d)
    a = rt.Attention(4, 1, d, max_seqs=1024)
    check_shared(rt, a, t, pools, dense, 1, 4, 1, d, "bf16", slots=list(range(1023)) + [5])
    t, pools, dense = pool_of(rt, [70000, 3], 0, 1, d, "bf16", 1024, d)
    check_shared(rt, a, t, pools, dense, 0, 4, 1, d, "bf16", slots=[0, 1, 0])


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("window", [0, 50])
def test_hidden_numbers_that_are_not_finite(rt, d, window):
    """Infinities and NaNs among keys, values and queries reach the rows that see them, and no others."""
    lens, heads, kvh = [200, 170], 4, 2
    q, k, v, offsets = packed(lens, heads, kvh, d, "bf16", d)
    clean = v.clone()
    v[40, 0, 5], v[41, 0, 5], v[131, 1, d - 1], v[260, 0] = math.inf, -math.inf, math.nan, math.nan
    kk = k.clone()
    kk[150, 1, 3], kk[199, 0, 0] = math.nan, math.inf
    qq = q.clone()
    qq[7, 3, 0] = math.nan
    a = rt.Attention(heads, kvh, d, max_seqs=2)
    out = a.prompt(qq, kk, v, i32(offsets), window=window)
    assert a.device_error() == (0, 0)
    for x, y in zip(offsets, offsets[1:]):
        want, _ = acc.attend(q[x:y], k[x:y], clean[x:y], None, window)
        for h in range(heads):
            for i in range(y - x):
                first = max(0, i - window + 1) if window else 0
                see = slice(x + first, x + i + 1)
                o, w = out[x + i, h].double(), want[i, h]
                if torch.isnan(qq[x + i, h]).any() or not torch.isfinite(kk[see, h // 2]).all():
                    # a NaN score spoils the row; an infinite one may leave a single weight
                    assert not torch.isfinite(o).all() or torch.isinf(kk[see, h // 2]).any()
                    continue
                bad = ~torch.isfinite(v[see, h // 2]).all(0)
                assert (~torch.isfinite(o[bad])).all() and torch.isfinite(o[~bad]).all()
                if not bad.all():
                    err = (o - w)[~bad].norm() / w[~bad].norm()
                    assert err <= limit("bf16", d, min(i + 1, window or i + 1)), (x, i, h, err)


@pytest.mark.parametrize("d", [64, 256])
def test_strides_and_given_outputs(rt, d):
    """Projections packed in one tensor, heads before rows, an output in between others and one that is not aligned."""
    lens, heads, kvh = [150, 1, 77], 4, 2
    n = sum(lens)
    g = torch.Generator().manual_seed(d)
    wide = torch.randn(n, heads + 2 * kvh, d, generator=g).bfloat16().cuda()
    q, k, v = wide[:, :heads], wide[:, heads:heads + kvh], wide[:, heads + kvh:]
    offsets = [0, 150, 151, 228]
    a = rt.Attention(heads, kvh, d, max_seqs=3)
    plain = a.prompt(q.contiguous(), k.contiguous(), v.contiguous(), i32(offsets))
    check_prompt(plain, q, k, v, offsets, "bf16")
    assert torch.equal(a.prompt(q, k, v, i32(offsets)), plain)
    turned = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    assert torch.equal(a.prompt(*turned, i32(offsets)), plain)
    for pad in (1, 8, 16):
        big = torch.full((n + 4, heads + 1, d + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        out = big[2:2 + n, :heads, pad // 2:pad // 2 + d]
        assert a.prompt(q, k, v, i32([3, 150, 151, 200]), out=out) is out
        rest = a.prompt(q, k, v, i32([3, 150, 151, 200]))
        assert torch.equal(out[3:200], rest[3:200])
        assert (out[:3] == 7).all() and (out[200:] == 7).all() and not rest[:3].any() and not rest[200:].any()
        keep = torch.ones_like(big, dtype=torch.bool)
        keep[2:2 + n, :heads, pad // 2:pad // 2 + d] = False
        assert (big[keep] == 7).all()


@pytest.mark.parametrize("d", [64, 512])
@pytest.mark.parametrize("n", [5, 60])
def test_shared_strides_scale_and_given_outputs(rt, d, n):
    """Queries out of a packed projection, outputs between others and not aligned, another scale; 60 sequences of
    1,280 rows are attended to once, five on their own."""
    heads, kvh, page, shared = 8, 2, 64, 20
    lens = [shared * page + (13 * i) % 90 for i in range(n)]
    t, pools, dense = pool_of(rt, lens, shared, kvh, d, "bf16", page, d + n)
    a = rt.Attention(heads, kvh, d, max_seqs=n)
    wide = torch.randn(n, heads + 4, d, generator=torch.Generator().manual_seed(n)).bfloat16().cuda()
    q, slots = wide[:, 2:2 + heads], i32(list(range(n)))
    plain = a.shared(q.contiguous(), *pools, t, slots, shared, scale=0.05)
    for i, (k, v) in enumerate(dense):
        right(plain[i:i + 1], acc.attend(q[i:i + 1], k, v, 0.05)[0], "bf16", len(k))
    for pad in (0, 1, 8):
        big = torch.full((n, heads + 1, d + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        out = big[:, 1:, pad // 2:pad // 2 + d]
        if pad == 1:
            out = big.flatten()[1:1 + n * heads * d].view(n, heads, d)
        assert a.shared(q, *pools, t, slots, shared, scale=0.05, out=out) is out
        assert torch.equal(out, plain)
        if pad != 1:
            assert (big[:, 0] == 7).all() and (pad == 0 or (big[:, 1:, pad // 2 + d:] == 7).all())


def test_scale(rt):
    q, k, v, offsets = packed([140], 4, 2, 128, "bf16", 3)
    a = rt.Attention(4, 2, 128, max_seqs=1)
    for scale in (0.02, 0.2):
        check_prompt(a.prompt(q, k, v, i32(offsets), scale=scale), q, k, v, offsets, "bf16", scale=scale)


@pytest.mark.parametrize("d", [64, 512])
def test_rising_scores(rt, d):
    """Each key's score is above all before it, by more than what raises the reference: the output follows every time."""
    t = 300
    q = torch.zeros(t, 2, d)
    q[:, :, 0] = 4.0
    k = torch.zeros(t, 1, d)
    k[:, 0, 0] = torch.arange(t) * 0.5
    v = torch.randn(t, 1, d, generator=torch.Generator().manual_seed(1))
    q, k, v = (x.bfloat16().cuda() for x in (q, k, v))
    a = rt.Attention(2, 1, d, max_seqs=1)
    check_prompt(a.prompt(q, k, v, i32([0, t]), scale=1.0), q, k, v, [0, t], "bf16", scale=1.0)
    check_prompt(a.prompt(q, k.flip(0), v, i32([0, t]), scale=1.0), q, k.flip(0), v, [0, t], "bf16", scale=1.0)


def test_many_sequences(rt):
    """More sequences than a warp looks at together, most of them empty or a token long."""
    g = torch.Generator().manual_seed(0)
    lens = [int(x) for x in torch.randint(0, 4, (1000,), generator=g)]
    lens[500:503] = [0, 333, 0]
    q, k, v, offsets = packed(lens, 3, 1, 64, "f16", 1, 2, 9)
    a = rt.Attention(3, 1, 64, dtype=torch.float16, max_seqs=1024)
    out = a.prompt(q, k, v, i32(offsets))
    assert a.device_error() == (0, 0)
    check_prompt(out, q, k, v, offsets, "f16")
    none = a.prompt(q[:5], k[:5], v[:5], i32([0] * 20))
    assert not none.any() and a.prompt(q[:0], k[:0], v[:0], i32([0, 0])).shape == (0, 3, 64)
    assert a.device_error() == (0, 0)


def test_offsets_that_are_wrong(rt):
    """Sequences whose offsets fall or leave the rows are passed over; the others are right."""
    q, k, v, _ = packed([60], 4, 2, 128, "bf16", 9)
    a = rt.Attention(4, 2, 128, max_seqs=8)
    for offsets, good in (([0, 20, 61], [(0, 20)]), ([-3, 10, 60], [(10, 60)]), ([0, 30, 20, 60], [(0, 30), (20, 60)]),
                          ([0, 1 << 30, 40, 50], [(40, 50)]), ([5, -1 << 31, 50, 60], [(50, 60)])):
        out = torch.full_like(q, 3.0)
        a.prompt(q, k, v, i32(offsets), out=out)
        assert a.device_error() == (-7, 2)
        if offsets == [0, 30, 20, 60]:       # rows of both: either's
            continue
        seen = torch.zeros(60, dtype=torch.bool)
        for x, y in good:
            want, _ = acc.attend(q[x:y], k[x:y], v[x:y])
            right(out[x:y], want, "bf16", list(range(1, y - x + 1)))
            seen[x:y] = True
        assert (out[~seen] == 3).all()


def test_slots_that_are_wrong(rt):
    """Each wrong sequence gets zeros and its error bit; the others are right."""
    heads, kvh, d, page, n = 8, 2, 128, 16, 6
    for shared in (2, 70):
        lens = [shared * page + x for x in (5, 40, 0, 17, 300, 9)]
        t, pools, dense = pool_of(rt, lens, shared, kvh, d, "bf16", page, shared)
        a = rt.Attention(heads, kvh, d, max_seqs=64)
        for wrong, bit in (("slot", 8), ("short", 2), ("long", 2), ("other", 2), ("missing", 2), ("outside", 2)):
            table, ln = t.table.clone(), t.lens.clone()
            slots = [0, 1, 2, 3, 4, 5] * (10 if shared > 2 else 1)     # (60 x 1,120 rows: attended to once)
            bad = 3
            if wrong == "slot":
                slots = [99 if s == 3 else s for s in slots]
                bad = 99
            elif wrong == "short":
                t.lens[3] = shared * page - 1
            elif wrong == "long":
                t.lens[3] = 1 << 21
            elif wrong == "other":
                t.table[3, 1] = table[3, shared]
            elif wrong == "missing":
                t.table[3, shared] = -1
            else:
                t.table[3, shared] = t.n_pages
            q = torch.randn(len(slots), heads, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
            out = a.shared(q, *pools, t, i32(slots), shared)
            assert a.device_error() == (-7, bit)
            for i, s in enumerate(slots):
                if s == bad:
                    assert not out[i].any()
                else:
                    right(out[i:i + 1], acc.attend(q[i:i + 1], *dense[s])[0], "bf16", len(dense[s][0]))
            t.table.copy_(table)
            t.lens.copy_(ln)


def test_pools_past_32_bits(rt):
    """Pages whose places in the pool pass 2^32 bytes and 2^31 elements."""
    kvh, d, page, pages = 8, 512, 64, 9000
    heads, n, shared = 16, 17, 18
    t = rt.PageTable(n + 2, pages, page, 8900)
    t.extend(i32([n + 1]), i32([8740 * page]), 0)          # the pool's first 8,740 pages: 2.29e9 elements
    pools = [torch.zeros(pages, kvh, page, d, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    g = torch.Generator().manual_seed(4)
    rows = t.extend(i32([n]), i32([shared * page]), shared * page)[0]
    x = [torch.randn(shared * page, kvh, d, generator=g).bfloat16().cuda() for _ in "kv"]
    t.store(*x, rows, *pools)
    t.share(i32(list(range(n))), n, shared)
    counts = [5 + i for i in range(n)]
    rows, offsets, _ = t.extend(i32(list(range(n))), i32(counts), sum(counts))
    assert int(rows.min()) * kvh * d > 2 ** 31
    y = [torch.randn(sum(counts), kvh, d, generator=g).bfloat16().cuda() for _ in "kv"]
    t.store(*y, rows, *pools)
    o = offsets.tolist()
    dense = [(torch.cat([x[0], y[0][o[i]:o[i + 1]]]), torch.cat([x[1], y[1][o[i]:o[i + 1]]])) for i in range(n)]
    a = rt.Attention(heads, kvh, d, max_seqs=n)
    check_shared(rt, a, t, pools, dense, shared, heads, kvh, d, "bf16")
    t.truncate(i32([n + 1]))
    check_shared(rt, a, t, pools, dense, shared, heads, kvh, d, "bf16")


def test_captured_replayed_and_on_streams(rt):
    """A graph replayed with other offsets, lengths and inputs in place; two objects on two streams at once."""
    lens = [90, 130]
    q, k, v, offsets = packed(lens, 8, 2, 128, "bf16", 5)
    a, b = rt.Attention(8, 2, 128, max_seqs=16), rt.Attention(8, 2, 128, max_seqs=16)
    off = i32(offsets)
    t, pools, dense = pool_of(rt, [40, 64, 33], 2, 2, 128, "bf16", 16, 3)
    slots, qd = i32([2, 0, 1]), torch.randn(3, 8, 128, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    a.prompt(q, k, v, off)
    a.shared(qd, *pools, t, slots, 2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o1 = a.prompt(q, k, v, off)
        o2 = a.shared(qd, *pools, t, slots, 2)
    for step, new in enumerate(([0, 90, 220], [10, 10, 200], [0, 1, 2], [0, 220, 220])):
        off.copy_(i32(new))
        slots.copy_(i32([step % 3, 1, 2]))
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(step)).to(q))
        graph.replay()
        check_prompt(o1, q, k, v, new, "bf16")
        for i, s in enumerate([step % 3, 1, 2]):
            right(o2[i:i + 1], acc.attend(qd[i:i + 1], *dense[s])[0], "bf16", len(dense[s][0]))
    assert a.device_error() == (0, 0)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    off.copy_(i32([0, 90, 220]))
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got += [a.prompt(q, k, v, off, stream=one), b.prompt(q, k, v, off, stream=two), a.shared(qd, *pools, t, slots, 2, stream=one),
                b.shared(qd, *pools, t, slots, 2, stream=two)]
    torch.cuda.synchronize()
    for x in got:
        assert torch.equal(x, got[0] if x.shape == got[0].shape else got[2])
    check_prompt(got[0], q, k, v, [0, 90, 220], "bf16")
    with pytest.raises(ValueError):
        a.prompt(q, k, v, i32([0, 4]).cpu())


def test_a_batch_from_prompt_to_release(rt):
    """As a program uses them: prompts behind one instruction attended to and stored, then steps of one token
    and rejected drafts, then all pages back."""
    heads, kvh, d, page, pre, n = 8, 2, 128, 16, 96, 5
    own = [1, 30, 17, 64, 45]
    t = rt.PageTable(n + 1, 200, page, 40)
    pools = [torch.full((200, kvh, page, d), math.nan, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    a = rt.Attention(heads, kvh, d, max_seqs=n + 1)
    q, k, v, _ = packed([pre + sum(own)], heads, kvh, d, "bf16", 1)
    starts = [pre + sum(own[:i]) for i in range(n)]
    idx = [torch.tensor(list(range(pre)) + list(range(s, s + m)), device="cuda") for s, m in zip(starts, own)]
    every = torch.cat(idx)
    offsets = [0]
    for x in idx:
        offsets.append(offsets[-1] + len(x))
    out = a.prompt(q[every], k[every], v[every], i32(offsets))
    check_prompt(out, q[every], k[every], v[every], offsets, "bf16")
    slots = i32([3, 0, 4, 1, 2])
    rows = t.extend(i32([n]), i32([pre]), pre)[0]
    t.store(k[:pre], v[:pre], rows, *pools)
    t.share(slots, n, pre // page)
    rows = t.extend(slots, i32(own), sum(own))[0]
    t.store(k[pre:], v[pre:], rows, *pools)
    held = [(k[x], v[x]) for x in idx]
    g = torch.Generator().manual_seed(9)
    for step in range(20):
        new = 3 if step % 4 == 1 else 1                         # some steps draft three tokens and keep one
        kn, vn = (torch.randn(n, new, kvh, d, generator=g).bfloat16().cuda() for _ in "kv")
        rows, _, lens = t.extend(slots, i32([new] * n), n * new)
        t.store(kn.flatten(0, 1), vn.flatten(0, 1), rows, *pools)
        if new > 1:
            t.truncate(slots, lens - (new - 1))
        held = [(torch.cat([x, kn[i, :1]]), torch.cat([y, vn[i, :1]])) for i, (x, y) in enumerate(held)]
        qn = torch.randn(n, heads, d, generator=g).bfloat16().cuda()
        out = a.shared(qn, *pools, t, slots, pre // page)
        for i, (x, y) in enumerate(held):
            right(out[i:i + 1], acc.attend(qn[i:i + 1], x, y)[0], "bf16", len(x))
    t.truncate(i32([5, 0, 1, 2, 3, 4]))
    assert (t.table == -1).all() and not t.lens.any()
    rows, _, lens = t.extend(i32([0, 1, 2, 3, 4]), i32([640] * 5), 3200)
    assert sorted(rows.tolist()) == list(range(3200)) and t.device_error() == (0, 0) and a.device_error() == (0, 0)


def test_refusals(rt):
    from accelerator_decode_gb300 import g4
    a = rt.Attention(4, 2, 64, max_seqs=2)
    q, k, v, _ = packed([8], 4, 2, 64, "bf16", 0)
    off = i32([0, 8])
    t = rt.PageTable(2, 4, 16, 2)
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    s = i32([0])
    for call in (lambda: a.prompt(q, k, v, i32([0, 2, 4, 8])), lambda: a.prompt(q, k, v, i32([0])), lambda: a.prompt(q, k, v, off, scale=-1.0),
                 lambda: a.prompt(q, k, v, off, scale=math.nan), lambda: a.prompt(q, k, v, off, window=-1),
                 lambda: a.prompt(q, k, v, off, out=q), lambda: a.prompt(q, k[:, :1].expand(8, 2, 64), v, off),
                 lambda: a.prompt(q, k, torch.zeros(8, 2, 68, dtype=torch.bfloat16, device="cuda")[..., :64], off),
                 lambda: a.prompt(torch.zeros(8, 4, 65, dtype=torch.bfloat16, device="cuda")[..., 1:], k, v, off),
                 lambda: a.prompt(q, k, v, off, out=torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda").expand(8, 4, 64)),
                 lambda: a.shared(q[:3], pool, pool, t, i32([0, 0, 0]), 0), lambda: a.shared(q[:1], pool, pool, t, s, 3),
                 lambda: a.shared(q[:1], pool, pool, t, s, -1), lambda: a.shared(q[:1], pool, pool, t, s, 0, out=q[:1])):
        with pytest.raises(g4.G4Error):
            call()
    assert not a.shared(q[:1], pool, pool, t, s, 0).any()
    assert a.device_error() == (0, 0)


def test_allocations_that_fail(rt, monkeypatch):
    """The allocation of each handle fails, for want of memory and injected: out of memory, and nothing is kept."""
    from accelerator_decode_gb300 import g4
    for make in (lambda: rt.PageTable(2, 4, 16, 2), lambda: rt.Attention(4, 2, 64, max_seqs=2)):
        monkeypatch.setenv("G4_FAIL_ALLOC_AT", "1")
        with pytest.raises(g4.G4Error) as e:
            make()
        assert e.value.status == g4.G4_ERR_OOM
        monkeypatch.delenv("G4_FAIL_ALLOC_AT")
        op = make()
        assert op.device_bytes() > 0
        op.close()
