// Host parts that the page table and the 16-bit attention share.
#pragma once
#include <algorithm>
#include <new>
#include <type_traits>

#include "host.h"
#include "pages_layout.h"

// Device memory of an op: one allocation, cut into arrays (with the allocation-failure injection of g4_create,
// G4_FAIL_ALLOC_AT).
struct g4_paged_memory {
  void* all = nullptr;
  size_t bytes = 0;
};

struct g4_pages {
  g4_pages_config cfg{};
  int device = 0, sms = 0;
  g4::Pages p{};
  g4_paged_memory mem;
};

namespace g4 {

// The arrays that `visit` names as take(&pointer, count): a first pass adds their sizes up, a second hands them out.
// The first `zeros` bytes, which hold the arrays named first, are cleared on `st`.
template <class Visit>
g4_status paged_alloc(g4_paged_memory* m, size_t zeros, cudaStream_t st, Visit visit) {
  size_t at = 0;
  char* base = nullptr;
  auto take = [&](auto** p, size_t count) {
    if (base) *p = reinterpret_cast<std::remove_reference_t<decltype(*p)>>(base + at);
    at += (std::max<size_t>(count, 1) * sizeof(**p) + 255) / 256 * 256;
  };
  visit(take);
  const char* fail = getenv("G4_FAIL_ALLOC_AT");
  if (fail && atoi(fail) == 1) return G4_ERR_OOM;  // injected
  const cudaError_t e = cudaMalloc(&m->all, at);
  if (e != cudaSuccess) {
    m->all = nullptr;
    cuda_ok(e, "cudaMalloc");
    cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? G4_ERR_OOM : G4_ERR_CUDA;
  }
  m->bytes = at;
  base = static_cast<char*>(m->all);
  at = 0;
  visit(take);
  CK(cudaMemsetAsync(m->all, 0, std::min(zeros, m->bytes), st));
  return G4_OK;
}

// A tensor argument [rows][heads][d] of 16-bit numbers.
struct Paged16 {
  uint16_t* p = nullptr;
  long row = 0, head = 0;
  int vec = 0;  // 16-byte accesses
};
inline bool paged_tensor(const g4_kv4_tensor* t, long rows, long heads, int d, bool written, Paged16* out) {
  if (!t || !t->data || reinterpret_cast<uintptr_t>(t->data) % 2) return false;
  struct { long stride, size; } ax[2] = {{(long)t->row_stride, rows}, {(long)t->head_stride, heads}};
  for (auto& x : ax)
    if (x.stride < 0 || x.stride > (1L << 46) / std::max(x.size, 1L)) return false;
  if (written) {  // no element twice
    if (ax[0].stride > ax[1].stride) std::swap(ax[0], ax[1]);
    long extent = d;
    for (auto& x : ax) {
      if (x.size <= 1) continue;
      if (x.stride < extent) return false;
      extent += x.stride * (x.size - 1);
    }
  }
  out->p = static_cast<uint16_t*>(t->data);
  out->row = t->row_stride;
  out->head = t->head_stride;
  out->vec = reinterpret_cast<uintptr_t>(t->data) % 16 == 0 && t->row_stride % 8 == 0 && t->head_stride % 8 == 0;
  return true;
}
inline bool paged_head_dim(int d) { return d == 64 || d == 128 || d == 256 || d == 512; }

// An op's error word, read and cleared.
inline g4_status paged_error(int device, int* err, g4_stream stream, int32_t* word_out) {
  DEVICE_GUARD(device);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int w = 0;
  CK(cudaMemcpyAsync(&w, err, sizeof(int), cudaMemcpyDeviceToHost, st));
  CK(cudaMemsetAsync(err, 0, sizeof(int), st));
  CK(cudaStreamSynchronize(st));
  if (word_out) *word_out = w;
  if (w & G4_DEV_TIMEOUT) return G4_ERR_TIMEOUT;
  return w ? G4_ERR_DEVICE_CHECK : G4_OK;
}

}  // namespace g4
