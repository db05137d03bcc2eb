// What lies where in a page table (pages.cuh), for the kernels that read it.
#pragma once
#include "common.cuh"

namespace g4 {

constexpr int kPagesMaxSlots = 1024;

struct Pages {
  int* table;  // [n_slots][max_pages]
  int* lens;   // [n_slots]
  int *refs, *owner, *free, *top;
  unsigned* ticket;
  int* err;
  int n_slots, n_pages, log_page, max_pages;
  __device__ __forceinline__ int page() const { return 1 << log_page; }
  __device__ __forceinline__ int capacity() const { return max_pages << log_page; }
  __device__ __forceinline__ int pages_of(int rows) const { return (rows + page() - 1) >> log_page; }
};

}  // namespace g4
