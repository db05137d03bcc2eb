"""Accounts with many sequences in a call: repeated slots are skipped wherever they stand, and finding
them costs no more than the attention itself."""
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


def cache(rt, n, keys, kvh, group, q_len, d, dtype):
    q, k, v = (x.cuda() for x in acc.inputs(n, keys, kvh, group, q_len, d, dtype, n))
    c = rt.KV4Cache(n, keys, kvh * group, kvh, d, max_q_len=q_len, track=True)
    c.append(k, v, i32(list(range(n))), i32([0] * n))
    return c, q


@pytest.mark.parametrize("n,kvh,group,q_len,d,dtype", [(1024, 1, 8, 1, 64, "bf16"), (300, 2, 8, 1, 256, "f32"),
                                                       (300, 1, 8, 17, 64, "bf16"), (330, 1, 8, 9, 256, "bf16"),
                                                       (520, 1, 4, 3, 512, "bf16"), (200, 1, 4, 3, 512, "f16")])
def test_repeated_slots_anywhere(rt, n, kvh, group, q_len, d, dtype):
    from accelerator_decode_gb300 import g4
    keys = 70
    c, q = cache(rt, n, keys, kvh, group, q_len, d, dtype)
    g = torch.Generator().manual_seed(n)
    slots = torch.randperm(n, generator=g)
    again = torch.randperm(n - 1, generator=g)[:n // 10] + 1       # these name an earlier one's slot
    for i in again.tolist():
        slots[i] = slots[int(torch.randint(0, i, (1,), generator=g))]
    first = {}
    for i, s in enumerate(slots.tolist()):
        first.setdefault(s, i)
    owner = torch.tensor([first[s] == i for i, s in enumerate(slots.tolist())])
    lens = torch.randint(q_len, keys + 1, (n,), generator=g).to(torch.int32).cuda()
    slots = slots.to(torch.int32).cuda()
    c.attend(q, slots, lens)
    assert c.device_error() == (0, 0)                              # reading a slot twice is fine
    # without the repeated ones the work is cut alike, so the bits are those of the call that skips them
    want = c.attend(q, slots, torch.where(owner.cuda(), lens, 0))
    out = c.attend(q, slots, lens, accumulate=True)
    assert c.device_error() == (g4.G4_ERR_DEVICE_CHECK, g4.G4_DEV_BAD_SLOT)
    assert torch.equal(out, want) and not out[~owner.cuda()].any()
    gained = c.account(i32(list(range(n))), i32([0] * n), keys)[1].sum(-1)   # [slot, head]
    named = torch.zeros(n, dtype=torch.bool)
    named[list(first)] = True
    assert not gained[~named.cuda()].any()
    whole = gained[named.cuda()]
    assert ((whole - q_len * group).abs() <= q_len * group * 2.0 ** -12).all()


def test_accounts_of_many_sequences_take_no_longer_than_their_attention(rt):
    c, q = cache(rt, 1024, 300, 8, 4, 1, 64, "bf16")
    slots, lens = i32(list(range(1024))), i32([300] * 1024)

    def time(accumulate):
        best = 1e9
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            c.attend(q, slots, lens, accumulate=accumulate)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    plain, account = time(False), time(True)
    assert account <= 8 * plain, (plain, account)                  # it was 300 times as long
    assert c.device_error() == (0, 0)
