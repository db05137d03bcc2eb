"""The decode step over 4-bit cache rows (kv_format int4) against the oracle, through the C ABI:
decode steps, prefill blocks, a binding sliding window, paged caches and long contexts at E2B head
dims, teacher-forced as the other cache variants are."""
import numpy as np
import pytest

import oracle
import synth
from test_gpu_kv import check, forced

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def rt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from accelerator_decode_gb300 import runtime
    return runtime


@pytest.mark.parametrize("name,fmt,page", [("tiny", "bf16", 0), ("tiny10", "w4a16", 0), ("tiny10", "w4a16", 16)])
def test_int4_kv_matches_oracle(rt, name, fmt, page):
    """Two sequences past the tiny configs' window of 64."""
    cfg = synth.get_config(name)
    w = synth.make_weights(cfg, fmt, seed=11, gain_std=0.1)
    prompts = synth.make_prompts(cfg["vocab"], 2, 70, seed=11)
    ref = oracle.Oracle(cfg, w, max_batch=2, max_context=96, kv_dtype="int4").generate(prompts, 10, keep_logits=True)
    dec = rt.Decoder(cfg, w, max_batch=2, max_context=96, kv_format="int4", kv_page_size=page)
    toks, logits = forced(dec, prompts, ref, paged=bool(page))
    assert dec.device_error() == (0, 0)
    dec.close()
    check(ref, toks, logits, f"int4 {name}/{fmt}/{page}")


def test_int4_kv_is_not_another_cache(rt):
    """The int4 run follows the int4 oracle more closely than the bf16 and int8 ones."""
    cfg = synth.get_config("tiny")
    w = synth.make_weights(cfg, "bf16", seed=4)
    prompts = synth.make_prompts(cfg["vocab"], 1, 20, seed=4)
    refs = {kv: oracle.Oracle(cfg, w, max_batch=1, max_context=64, kv_dtype=kv).generate(prompts, 10, keep_logits=True)
            for kv in ("bf16", "int8", "int4")}
    dec = rt.Decoder(cfg, w, max_batch=1, max_context=64, kv_format="int4")
    _, logits = forced(dec, prompts, refs["int4"])
    first = {kv: float(np.max(np.abs(logits[0] - r["logits"][0]))) for kv, r in refs.items()}
    assert 10 * first["int4"] < min(first["bf16"], first["int8"]), first
    assert dec.device_error() == (0, 0)
    dec.close()


@pytest.mark.parametrize("batch", [1, 6, 9])
def test_int4_kv_long_context_e2b_heads(rt, batch):
    """Head dims 256 / 512, window 512 binding, 600 tokens; the staged step and the GEMM's."""
    cfg = synth.get_config("mid")
    w = synth.make_weights(cfg, "w4a16", seed=0, qk_gain=0.5)
    prompts = synth.make_prompts(cfg["vocab"], batch, 600, seed=0)
    if batch > 1:
        prompts = [p[:600 - 61 * i] for i, p in enumerate(prompts)]
    ref = oracle.Oracle(cfg, w, max_batch=batch, max_context=640, kv_dtype="int4")
    dec = rt.Decoder(cfg, w, max_batch=batch, max_context=640, kv_format="int4", kv_page_size=128 if batch == 9 else 0)
    if batch == 1:
        r = ref.generate(prompts, 4, keep_logits=True)
        toks, logits = forced(dec, prompts, r)
        check(r, toks, logits, "int4 mid 600")
    else:
        nxt, lg = dec.prefill(list(range(batch)), prompts, want_logits=True)
        torch.cuda.synchronize()
        for i in (0, batch - 1):          # sequences are independent: two of them against the oracle
            o = oracle.Oracle(cfg, w, max_batch=1, max_context=640, kv_dtype="int4")
            r = o.generate([prompts[i]], 1, keep_logits=True)
            assert float(np.max(np.abs(lg[i].cpu().numpy() - r["logits"][0][0]))) <= 3e-2
        pos = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
        if batch == 9:
            for i, p in enumerate(prompts):
                dec.reserve(i, len(p) + 1)
        tok, out = nxt.clone(), torch.empty(batch, dtype=torch.int32, device="cuda")
        lgt = torch.empty(batch, cfg["vocab"], dtype=torch.float32, device="cuda")
        dec.decode_step(torch.arange(batch, dtype=torch.int32, device="cuda"), tok, pos, out, lgt)
        torch.cuda.synchronize()
        for i in (0, batch - 1):
            o = oracle.Oracle(cfg, w, max_batch=1, max_context=640, kv_dtype="int4")
            r = o.generate([np.concatenate([prompts[i], tok[i:i + 1].cpu().numpy()])], 1, keep_logits=True)
            assert float(np.max(np.abs(lgt[i].cpu().numpy() - r["logits"][0][0]))) <= 3e-2
    assert dec.device_error() == (0, 0)
    dec.close()


def test_int4_kv_errors_and_modes(rt):
    """Bad positions and missing pages are reported, the sequence beside is right, the cache has the
    bytes it should, and the persistent step refuses these rows."""
    from accelerator_decode_gb300 import g4
    cfg = synth.get_config("tiny")
    w = synth.make_weights(cfg, "bf16", seed=2)
    prompts = synth.make_prompts(cfg["vocab"], 2, 30, seed=2)
    dec = rt.Decoder(cfg, w, max_batch=2, max_context=64, kv_format="int4", kv_page_size=16)
    with pytest.raises(g4.G4Error):
        dec.set_step_mode(1)
    nxt, _ = dec.prefill([0, 1], prompts)
    slots, out = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    lg = torch.empty(2, cfg["vocab"], dtype=torch.float32, device="cuda")
    ok = torch.empty_like(lg)
    pos = torch.tensor([30, 30], dtype=torch.int32, device="cuda")
    dec.decode_step(slots, nxt, pos, out, ok)
    assert dec.device_error() == (0, 0)
    for bad in (64, -1, 50):                      # outside the context; on a page nobody reserved
        pos = torch.tensor([30, bad], dtype=torch.int32, device="cuda")
        dec.decode_step(slots, nxt, pos, out, lg)
        torch.cuda.synchronize()
        status, word = dec.device_error()
        assert status == g4.G4_ERR_DEVICE_CHECK and word & g4.G4_DEV_BAD_POSITION
        assert torch.equal(lg[0], ok[0])
    dec.close()
    size = {}
    for kv in ("bf16", "int4"):
        for ctx in (64, 64 + 4096):
            d = rt.Decoder(cfg, w, max_batch=2, max_context=ctx, kv_format=kv)
            size[kv, ctx] = d.device_bytes()
            d.close()
    # what else grows with the context (RoPE tables, attention splits) is the same in both
    saved = ((size["bf16", 64 + 4096] - size["int4", 64 + 4096]) - (size["bf16", 64] - size["int4", 64])) / (2 * 4096)
    assert saved == oracle.kv_bytes_per_token(cfg) - oracle.kv_bytes_per_token(cfg, kv_dtype="int4")
