"""The accuracy checks of the 4-bit cache's attention can fail: results that are wrong in a small way
are told from the right one rounded once, on the inputs of the GPU tests and without a GPU."""
import pytest

import kv4_accuracy as acc
import kv4_ref as ref
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d,q_len,keys", [(64, 1, 200), (128, 9, 700), (256, 1, 700), (512, 1, 700), (256, 33, 130), (64, 1, 4099)])
def test_wrong_results_are_told(dtype, d, q_len, keys):
    kvh, group = 2, 4
    q, k, v = acc.inputs(1, keys, kvh, group, q_len, d, dtype, d + keys)
    q, k, v = q[0], *(torch.from_numpy(ref.values(x[0].double().numpy())) for x in (k, v))
    want, gain = acc.attend(q, k, v)
    typ = acc.TYPES[dtype]
    good = lambda x: acc.right(x.to(typ), want, dtype, keys)
    assert good(want)
    assert not good(torch.zeros_like(want))
    assert not good(acc.attend(q, k, v.flip(0))[0])
    missing = acc.attend(q[-1:], k[:-1], v[:-1])[0]                # the newest key left out
    assert not acc.right(missing.to(typ), want[-1:], dtype, keys)
    w = keys // 2
    seen = acc.attend(q, k, v, window=w)[0]
    assert acc.right(seen.to(typ), seen, dtype, keys)
    for off in (w - 1, w + 1):
        assert not acc.right(acc.attend(q, k, v, window=off)[0].to(typ), seen, dtype, keys)
    if dtype != "bf16":                                            # queries cut to one bf16 part
        assert not good(acc.attend(q.bfloat16(), k, v)[0])
    ok = lambda x: acc.gains_right(x, gain, dtype, d)
    assert ok(gain.float()) and not ok(torch.zeros_like(gain)) and not ok(gain.flip(-1))
    lost = gain.clone()
    lost[:, -16:] = 0                                              # one block of keys without its weights
    assert not ok(lost)
