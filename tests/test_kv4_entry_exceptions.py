"""No C++ exception leaves a C entry: with every host allocation failing in turn, g4_kv4_create still
answers with a status (a C program that links the library and brings an operator new of its own)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HARNESS = r"""
#include "g4.h"
#include <cstdio>
#include <cstdlib>
#include <new>
static long left = -1;  // allocations until one fails; -1: none does
static bool failed = false;
void* operator new(size_t n) {
  if (left == 0) { failed = true; throw std::bad_alloc(); }
  if (left > 0) --left;
  if (void* p = malloc(n)) return p;
  throw std::bad_alloc();
}
void* operator new(size_t n, const std::nothrow_t&) noexcept {
  if (left == 0) { failed = true; return nullptr; }
  if (left > 0) --left;
  return malloc(n);
}
void operator delete(void* p) noexcept { free(p); }
void operator delete(void* p, size_t) noexcept { free(p); }
int main() {
  g4_kv4_config c{4, 100, 8, 2, 64, 8, 0, 0, 1};
  int out = 0, hits = 0;
  for (int n = 0; n < 40; ++n) {
    g4_kv4* op = reinterpret_cast<g4_kv4*>(1);
    failed = false;
    left = n;
    try {
      const g4_status s = g4_kv4_create(0, &c, nullptr, &op);
      left = -1;
      if (failed && s == G4_OK && n == 0) ++out;
      if (s != G4_OK && op) ++out;
      if (s == G4_OK) g4_kv4_free(op);
    } catch (...) {
      left = -1;
      ++out;
    }
    hits += failed;
  }
  printf("%d %d\n", out, hits > 0);
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_failing_host_allocations(tmp_path):
    from accelerator_decode_gb300 import build
    build.build()
    src, exe = tmp_path / "h.cpp", tmp_path / "h"
    src.write_text(HARNESS)
    where = os.path.dirname(build.LIB)
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "include"), str(src), build.LIB, "-Wl,-rpath," + where,
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.split() == ["0", "1"], (r.returncode, r.stdout, r.stderr)
