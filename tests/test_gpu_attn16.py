"""Attention over 16-bit keys and values on the GPU against 64 bits (kv4_accuracy.attend).

Errors are taken per output row as |error| / |row| (kv4_accuracy explains why rows are sums of many
independent errors).  With u = eps / 2 of the type, an output row is off by
* its own rounding: 0.65 u in the root mean square, at most u (`few`);
* its weights' rounding into the products: each weight is off by at most u of itself, independently
  of the others, which moves the row as its own rounding does: 0.65 u, or for a row of few keys at most
  u sum p |v| / |sum p v|, which for the random values here (angles near a right one) is below 1.5 u;
  fp16 weights below 2^-14 are off by up to 2^-25 each, and n of them by 2^-25 sqrt(n) of a value;
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
