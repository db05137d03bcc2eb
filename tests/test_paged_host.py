"""What the page table and the 16-bit attention refuse before any device work (no GPU needed)."""
import ctypes
import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rt():
    from accelerator_decode_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from accelerator_decode_gb300 import runtime
    return runtime


@pytest.fixture(scope="module")
def g4(rt):
    return rt._g4


BAD, NOT = -1, -2      # INVALID_ARG, UNSUPPORTED


@pytest.mark.parametrize("sizes,want", [
    ((0, 4, 16, 2), BAD), ((2, 0, 16, 2), BAD), ((2, 4, 0, 2), BAD), ((2, 4, 16, 0), BAD), ((2, 4, -16, 2), BAD),
    ((1025, 4, 16, 2), NOT), ((2, 4, 8, 2), NOT), ((2, 4, 48, 2), NOT), ((2, 4, 16, (1 << 16) + 1), NOT),
    ((2, 1 << 27, 16, 2), NOT), ((2, 4, 1 << 20, 2), NOT)])
def test_page_table_sizes(g4, sizes, want):
    c, h, some = g4.g4_pages_config(*sizes), ctypes.c_void_p(5), ctypes.c_void_p(64)
    assert g4.lib.g4_pages_create(0, ctypes.byref(c), some, some, ctypes.byref(h)) == want
    assert h.value is None


@pytest.mark.parametrize("sizes,want", [
    ((0, 1, 64, 1, 1), BAD), ((4, 0, 64, 1, 1), BAD), ((5, 2, 64, 1, 1), BAD), ((4, 2, 64, 1, 0), BAD), ((-4, -2, 64, 1, 1), BAD),
    ((65, 1, 64, 1, 1), NOT), ((65, 65, 64, 1, 1), NOT), ((4, 2, 96, 1, 1), NOT), ((4, 2, 0, 1, 1), NOT), ((4, 2, 64, 0, 1), NOT),
    ((4, 2, 64, 3, 1), NOT), ((4, 2, 64, 1, 1025), NOT)])
def test_attention_sizes(g4, sizes, want):
    c, h = g4.g4_attn_config(*sizes), ctypes.c_void_p(5)
    assert g4.lib.g4_attn_create(0, ctypes.byref(c), ctypes.byref(h)) == want
    assert h.value is None


def test_null_arguments(g4):
    lib, c, a, p = g4.lib, g4.g4_pages_config(2, 4, 16, 2), g4.g4_attn_config(4, 2, 64, 1, 1), ctypes.c_void_p(64)
    h, t = ctypes.c_void_p(), ctypes.byref(g4.g4_kv4_tensor())
    assert lib.g4_pages_create(0, ctypes.byref(c), p, p, None) == BAD
    for args in ((None, p, p), (ctypes.byref(c), None, p), (ctypes.byref(c), p, None)):
        assert lib.g4_pages_create(0, *args, ctypes.byref(h)) == BAD
    assert lib.g4_pages_extend(None, None, 1, p, p, 1, p, p, p) == BAD
    assert lib.g4_pages_share(None, None, 1, p, 0, 1) == BAD
    assert lib.g4_pages_truncate(None, None, 1, p, p) == BAD
    assert lib.g4_pages_store(None, None, 1, p, 1, 64, t, t, p, p) == BAD
    assert lib.g4_pages_get_device_error(None, None, None) == BAD
    assert lib.g4_attn_create(0, None, ctypes.byref(h)) == BAD
    assert lib.g4_attn_create(0, ctypes.byref(a), None) == BAD
    assert lib.g4_attn_prompt(None, None, 1, p, 1, 0.0, 0, 0, t, t, t, t) == BAD
    assert lib.g4_attn_shared(None, None, None, 1, p, 0, 0.0, p, p, t, t) == BAD
    assert lib.g4_attn_get_device_error(None, None, None) == BAD
    assert lib.g4_pages_bytes(None) == 0 and lib.g4_attn_bytes(None) == 0
    lib.g4_pages_free(None)
    lib.g4_attn_free(None)


LONG = [2 ** 31, 2 ** 32 + 1, -2 ** 31 - 1]


@pytest.mark.parametrize("v", LONG)
def test_numbers_that_32_bits_do_not_hold(rt, v):
    for name in ("n_slots", "n_pages", "page_size", "max_pages"):
        with pytest.raises(ValueError, match="32 bits"):
            rt.PageTable(**{**dict(n_slots=2, n_pages=4, page_size=16, max_pages=2), name: v}, device=0)
    for name in ("num_q_heads", "num_kv_heads", "head_dim", "max_seqs"):
        with pytest.raises(ValueError, match="32 bits"):
            rt.Attention(**{**dict(num_q_heads=2, num_kv_heads=1, head_dim=64), name: v}, device=0)


class Spy:
    """Stands for the library: every call is noted and refused."""

    def __getattr__(self, name):
        def f(*a):
            raise AssertionError(f"{name} was called")
        return f


@pytest.fixture()
def ops(rt, monkeypatch):
    """A table and an attention without a device (CPU tensors have get_device() -1)."""
    t, a = object.__new__(rt.PageTable), object.__new__(rt.Attention)
    for o in (t, a):
        o.index, o.device, o.h = -1, torch.device("cpu"), None
        o._t = [rt._g4.g4_kv4_tensor() for _ in range(4)]
        o._p = [ctypes.byref(x) for x in o._t]
        o._stream = lambda stream: 0
    t.n_slots, t.n_pages, t.page_size, t.max_pages = 2, 4, 16, 2
    a.num_q_heads, a.num_kv_heads, a.head_dim, a.dtype = 4, 2, 64, torch.bfloat16
    monkeypatch.setattr(rt._g4, "lib", Spy())
    return t, a


def test_arguments(rt, ops):
    t, a = ops
    s = torch.zeros(2, dtype=torch.int32)
    q, k = torch.zeros(3, 4, 64).bfloat16(), torch.zeros(3, 2, 64).bfloat16()
    pool = torch.zeros(4, 2, 16, 64).bfloat16()
    rows = torch.zeros(3, dtype=torch.int32)
    q2 = torch.zeros(2, 4, 64).bfloat16()
    for v in LONG:
        for call in (lambda: t.extend(s, s, v), lambda: t.share(s, v, 1), lambda: t.share(s, 0, v),
                     lambda: a.prompt(q, k, k, s, window=v), lambda: a.shared(q2, pool, pool, t, s, v)):
            with pytest.raises(ValueError, match="32 bits"):
                call()
    for call, kind in (
            (lambda: t.extend(s, s, 1.5), TypeError), (lambda: t.extend(s, s[:1], 1), ValueError),
            (lambda: t.extend(s.long(), s, 1), TypeError), (lambda: t.extend(torch.zeros(4, dtype=torch.int32)[::2], s, 1), ValueError),
            (lambda: t.truncate(s, s[:1]), ValueError),
            (lambda: t.store(q, k, rows, pool, pool), ValueError), (lambda: t.store(k, k, rows, pool, pool.half()), TypeError),
            (lambda: t.store(k, k, rows.long(), pool, pool), TypeError), (lambda: t.store(k[0], k[0], rows, pool, pool), TypeError),
            (lambda: t.store(k, k, rows, pool.transpose(1, 2), pool), ValueError),
            (lambda: a.prompt(q, q, k, s), ValueError), (lambda: a.prompt(q.float(), k, k, s), TypeError),
            (lambda: a.prompt(q[0], k, k, s), ValueError), (lambda: a.prompt(q, k, k.half(), s), TypeError),
            (lambda: a.prompt(q, k, k, s.long()), TypeError), (lambda: a.prompt(q, k, k, s, out=q[:2]), ValueError),
            (lambda: a.prompt(q, k, k, s, out=q.half()), TypeError), (lambda: a.prompt(q, k, k, s, window=1.5), TypeError),
            (lambda: a.shared(q, pool, pool, t, s, 1), ValueError), (lambda: a.shared(q2, pool[:3], pool, t, s, 1), ValueError),
            (lambda: a.shared(q2, pool, pool.half(), t, s, 1), TypeError), (lambda: a.shared(q2, pool, pool, t, s.long(), 1), TypeError)):
        with pytest.raises(kind):
            call()
    with pytest.raises(TypeError):
        rt.Attention(4, 2, 64, dtype=torch.float32, device=0)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no gcc")
def test_struct_layout_matches_c(g4, tmp_path):
    src = tmp_path / "sz.c"
    src.write_text('#include "g4.h"\n#include <stdio.h>\n#include <stddef.h>\n'
                   'int main(void){printf("%zu %zu %zu %zu %d\\n", sizeof(g4_pages_config), offsetof(g4_pages_config, max_pages), '
                   'sizeof(g4_attn_config), offsetof(g4_attn_config, max_seqs), G4_DEV_NO_PAGES);return 0;}\n')
    exe = tmp_path / "sz"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = list(map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()))
    assert got == [ctypes.sizeof(g4.g4_pages_config), g4.g4_pages_config.max_pages.offset, ctypes.sizeof(g4.g4_attn_config),
                   g4.g4_attn_config.max_seqs.offset, g4.G4_DEV_NO_PAGES]
