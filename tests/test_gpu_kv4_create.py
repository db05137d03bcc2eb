"""g4_kv4_create that runs out of memory: an error, and every byte given back."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_allocation_failure_returns_oom_and_frees_everything(monkeypatch):
    from accelerator_decode_gb300 import g4, runtime

    def cache():
        return runtime.KV4Cache(8, 20000, 16, 2, 256, max_q_len=64, track=True)

    c = cache()                                        # warm: context, attributes
    size = c.device_bytes()
    c.close()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    free0 = torch.cuda.mem_get_info()[0]
    failed = 0
    for n in range(1, 40):
        monkeypatch.setenv("G4_FAIL_ALLOC_AT", str(n))
        try:
            c = cache()
        except g4.G4Error as e:
            assert e.status == g4.G4_ERR_OOM
            failed += 1
        else:
            assert c.device_bytes() == size
            c.close()
        torch.cuda.synchronize()
        assert abs(torch.cuda.mem_get_info()[0] - free0) <= 4 << 20, n
    assert 10 <= failed < 39
    monkeypatch.delenv("G4_FAIL_ALLOC_AT")
    cache().close()
