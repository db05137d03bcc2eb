"""The 4-bit KV cache without a GPU: the layout's addresses (the header the kernels use, compiled
for the host), refusals of bad arguments, and the reference's own borders."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import kv4_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "accelerator_decode_gb300", "csrc")


@pytest.fixture(scope="module")
def g4():
    from accelerator_decode_gb300 import build
    if not os.path.exists(build.LIB):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("libg4.so not built and no nvcc")
        build.build()
    from accelerator_decode_gb300 import g4 as mod
    return mod


LAYOUT = r"""
#include "kv4_layout.h"
#include <cstdio>
#include <vector>
using namespace g4;
template <int D> int check() {
  // every byte of a block belongs to exactly one number or scale (values: two nibbles a byte)
  std::vector<int> used(18 * D, 0);
  for (int r = 0; r < 16; ++r) {
    for (int o = 0; o < D / 8; ++o) for (int b = 0; b < 4; ++b) used.at(Kv4Off<D>::k_word(r, o) + b)++;
    for (int u = 0; u < D / 4; ++u) for (int b = 0; b < 2; ++b) used.at(Kv4Off<D>::v_half(r, u) + b)++;
    for (int g = 0; g < D / 32; ++g) for (int b = 0; b < 2; ++b) {
      used.at(Kv4Off<D>::k_scale(r, g) + b)++;
      used.at(Kv4Off<D>::v_scale(r, g) + b)++;
    }
  }
  for (int x : used) if (x != 1) return 1;
  // the fragments: lane 4g + t, word w of rows g and g + 8 holds numbers t D/4 + 8w ..
  for (int g = 0; g < 8; ++g) for (int t = 0; t < 4; ++t) for (int w = 0; w < D / 32; ++w)
    for (int hi = 0; hi < 2; ++hi) {
      const int piece = (w / 2 * 32 + 4 * g + t) * 16 + (2 * hi + w % 2) * 4;
      if (Kv4Off<D>::k_word(g + 8 * hi, (t * (D / 4) + 8 * w) / 8) != piece) return 2;
      for (int odd = 0; odd < 2; ++odd)
        if (Kv4Off<D>::v_half(2 * (t + 4 * hi) + odd, (g * (D / 8) + 4 * w) / 4) != 9 * D + piece + 2 * odd) return 3;
    }
  return 0;
}
int main() {
  const int bad = check<64>() * 1000 + check<128>() * 100 + check<256>() * 10 + check<512>();
  // page lookups: pages out of the pool and negative entries are no page; blocks of a page follow
  // one another per head; the last page may be partial
  int table[2 * 3] = {2, -1, 7, 0, 6, 1};
  Kv4Cache c{};
  c.table = table; c.log_bpp = 2; c.bpp = 4; c.max_pages = 3; c.n_pages = 7; c.n_slots = 2; c.capacity = 150; c.kvh = 2;
  int wrong = 0;
  for (int s = 0; s < 2; ++s) for (int h = 0; h < 2; ++h) for (int b = 0; b < 12; ++b) {
    const int pg = table[s * 3 + b / 4];
    const long want = pg < 0 || pg >= 7 ? -1 : (pg * 2 + h) * 4 + b % 4;
    wrong += kv4_block(c, s, h, b) != want;
  }
  c.table = nullptr; c.bpp = 10; c.kvh = 3;
  wrong += kv4_block(c, 4, 2, 9) != (4 * 3 + 2) * 10 + 9;
  // offsets past 32 bits
  c.bpp = 65536; c.kvh = 64;
  wrong += kv4_block(c, 1023, 63, 65535) * 16L * 1024 != ((1023L * 64 + 63) * 65536 + 65535) * 16 * 1024;
  printf("%d %d\n", bad, wrong);
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_layout_addresses(tmp_path):
    src = tmp_path / "layout.cpp"
    src.write_text(LAYOUT)
    exe = tmp_path / "layout"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined,address", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split() == ["0", "0"]


def test_config_layout_matches_c(g4, tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no gcc")
    src = tmp_path / "sz.c"
    src.write_text('#include "g4.h"\n#include <stdio.h>\n#include <stddef.h>\n'
                   'int main(void){printf("%zu %zu %zu %zu\\n", sizeof(g4_kv4_config), sizeof(g4_kv4_tensor), '
                   'offsetof(g4_kv4_config, track), offsetof(g4_kv4_tensor, head_stride));return 0;}\n')
    exe = tmp_path / "sz"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = list(map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()))
    assert got == [ctypes.sizeof(g4.g4_kv4_config), ctypes.sizeof(g4.g4_kv4_tensor), g4.g4_kv4_config.track.offset,
                   g4.g4_kv4_tensor.head_stride.offset]


GOOD = dict(n_slots=4, capacity=100, num_q_heads=8, num_kv_heads=2, head_dim=64, max_q_len=8, page_size=0, n_pages=0,
            track=0)


@pytest.mark.parametrize("change,status", [
    (dict(n_slots=0), "INVALID_ARG"), (dict(capacity=0), "INVALID_ARG"), (dict(num_kv_heads=3), "INVALID_ARG"),
    (dict(num_q_heads=0), "INVALID_ARG"), (dict(max_q_len=0), "INVALID_ARG"), (dict(track=2), "INVALID_ARG"),
    (dict(page_size=-16), "INVALID_ARG"), (dict(page_size=16), "INVALID_ARG"),     # no page table
    (dict(n_slots=1025), "UNSUPPORTED"), (dict(capacity=(1 << 20) + 1), "UNSUPPORTED"),
    (dict(head_dim=96), "UNSUPPORTED"), (dict(head_dim=0), "UNSUPPORTED"), (dict(max_q_len=65), "UNSUPPORTED"),
    (dict(num_kv_heads=65, num_q_heads=65), "UNSUPPORTED"), (dict(num_kv_heads=1, num_q_heads=65), "UNSUPPORTED"),
])
def test_create_refuses(g4, change, status):
    """Refused on the host, before any device call (so this runs without a GPU)."""
    c = g4.g4_kv4_config(**{**GOOD, **change})
    h = ctypes.c_void_p(1)
    assert g4.lib.g4_kv4_create(0, ctypes.byref(c), None, ctypes.byref(h)) == getattr(g4, "G4_ERR_" + status)
    assert h.value is None


@pytest.mark.parametrize("page", [8, 24, 100])
def test_create_refuses_page_sizes(g4, page):
    c = g4.g4_kv4_config(**{**GOOD, "page_size": page, "n_pages": 50})
    table = (ctypes.c_int32 * 64)()
    h = ctypes.c_void_p()
    assert g4.lib.g4_kv4_create(0, ctypes.byref(c), ctypes.cast(table, ctypes.c_void_p), ctypes.byref(h)) == \
        g4.G4_ERR_UNSUPPORTED


def test_null_handles_are_refused(g4):
    lib, bad = g4.lib, g4.G4_ERR_INVALID_ARG
    h = ctypes.c_void_p()
    assert lib.g4_kv4_create(0, None, None, ctypes.byref(h)) == bad
    assert lib.g4_kv4_create(0, ctypes.byref(g4.g4_kv4_config(**GOOD)), None, None) == bad
    t = g4.g4_kv4_tensor()
    assert lib.g4_kv4_append(None, None, 1, None, None, None, 1, ctypes.byref(t), ctypes.byref(t), None, None) == bad
    assert lib.g4_kv4_read(None, None, 1, None, None, None, 1, 0, ctypes.byref(t), None) == bad
    assert lib.g4_kv4_account(None, None, 1, None, None, None, 1, 0, None, None) == bad
    assert lib.g4_kv4_attend(None, None, 1, None, None, 1, None, 0.0, 0, 0, 0, ctypes.byref(t), ctypes.byref(t)) == bad
    assert lib.g4_kv4_evict(None, None, 1, None, None, 1, 0, None) == bad
    assert lib.g4_kv4_get_device_error(None, None, None) == bad
    assert lib.g4_kv4_bytes(None) == 0
    lib.g4_kv4_free(None)


def test_reference_borders():
    """The reference's rounding, by hand: ties to even, the clip, a zero group, one scale per 32."""
    x = np.zeros(64)
    x[:8] = [7, -7, 0.5, 1.5, 2.5, -3.5, 6.5, 0.49]
    c, s = ref.code_rows(x)
    assert s.tolist() == [1.0, 0.0]
    assert c[:8].tolist() == [7, -7, 0, 2, 2, -4, 6, 0] and not c[8:].any()
    assert ref.bf16_round(1 + 2.0 ** -8) == 1.0 and ref.bf16_round(1 + 3 * 2.0 ** -8) == 1 + 2.0 ** -6
    assert ref.bf16_round(2.0 ** -134) == 0.0 and ref.bf16_round(3 * 2.0 ** -134) == 2.0 ** -132
    assert ref.evict_source(np.array([0, 1, 2, 3]), np.array([1., 1., 0., 1.]), 2, 1).tolist() == [0, 3]


def test_oracle_rows_are_the_formats():
    """The decode oracle's 4-bit rows and the reference of the cache's operators, written apart."""
    from oracle import kv_int4_values
    g = np.random.default_rng(2)
    x = (g.standard_normal((50, 128)) * np.exp(g.uniform(-20, 20, (50, 1)))).astype(np.float32)
    x[3, 32:64] = 0
    x[4, :32] = np.clip(np.arange(-16, 16) * 0.5, -7, 7)   # a scale of one: ties
    np.testing.assert_array_equal(kv_int4_values(x, np.float64), ref.values(x))
