// C entry points of the page table (include/g4.h, g4_pages_*).
#include "paged_host.h"
#include "pages.cuh"

using namespace g4;

namespace {

bool pages_count(const g4_pages* op, int n_seq) { return n_seq >= 1 && n_seq <= op->cfg.n_slots; }

// Whether n and m int32 numbers share none.
bool pages_apart(const int32_t* a, long n, const int32_t* b, long m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return n <= 0 || m <= 0 || x + 4 * n <= y || y + 4 * m <= x;
}

__global__ void pages_init_kernel(const Pages p) {
  const long i = (long)blockIdx.x * blockDim.x + threadIdx.x, n = (long)gridDim.x * blockDim.x;
  for (long e = i; e < (long)p.n_slots * p.max_pages; e += n) p.table[e] = -1;
  for (long e = i; e < p.n_slots; e += n) p.lens[e] = 0;
  for (long e = i; e < p.n_pages; e += n) {
    p.free[e] = p.n_pages - 1 - (int)e;
    p.owner[e] = 0x7FFFFFFF;
  }
  if (i == 0) *p.top = p.n_pages;
}

g4_status pages_create_impl(g4_pages* op, cudaStream_t st) {
  Pages& p = op->p;
  TRY(paged_alloc(&op->mem, ~(size_t)0, st, [&](auto& take) {
    take(&p.top, 2 + kPagesCluster * kPagesThreads / 32);
    take(&p.ticket, 1);
    take(&p.err, 1);
    take(&p.refs, p.n_pages);
    take(&p.owner, p.n_pages);
    take(&p.free, p.n_pages);
  }));
  pages_init_kernel<<<op->sms, 256, 0, st>>>(p);
  CK(cudaGetLastError());
  return G4_OK;
}

}  // namespace

extern "C" {

g4_status g4_pages_create(int device, const g4_pages_config* cfg, int32_t* d_table, int32_t* d_lens, g4_pages** out) {
  if (!out) return G4_ERR_INVALID_ARG;
  *out = nullptr;
  if (!cfg || !d_table || !d_lens) return G4_ERR_INVALID_ARG;
  const g4_pages_config f = *cfg;
  if (f.n_slots < 1 || f.n_pages < 1 || f.page_size < 1 || f.max_pages < 1) return G4_ERR_INVALID_ARG;
  if (f.n_slots > kPagesMaxSlots || f.page_size < 16 || (f.page_size & (f.page_size - 1)) ||
      (long)f.max_pages * f.page_size > (1L << 20) || (long)f.n_pages * f.page_size >= (1L << 31))
    return G4_ERR_UNSUPPORTED;
  DEVICE_GUARD(device);
  g4_pages* op = new (std::nothrow) g4_pages();
  if (!op) return G4_ERR_OOM;
  op->cfg = f;
  op->device = device;
  op->p.table = d_table;
  op->p.lens = d_lens;
  op->p.n_slots = f.n_slots;
  op->p.n_pages = f.n_pages;
  op->p.max_pages = f.max_pages;
  while ((1 << op->p.log_page) < f.page_size) ++op->p.log_page;
  g4_status s = G4_ERR_CUDA;
  cudaStream_t st = nullptr;
  if (cuda_ok(cudaDeviceGetAttribute(&op->sms, cudaDevAttrMultiProcessorCount, device), "cudaDeviceGetAttribute") &&
      cuda_ok(cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking), "cudaStreamCreate")) {
    s = pages_create_impl(op, st);
    if (!cuda_ok(cudaStreamSynchronize(st), "cudaStreamSynchronize") && s == G4_OK) s = G4_ERR_CUDA;
    cudaStreamDestroy(st);
  }
  if (s != G4_OK) {
    cudaFree(op->mem.all);
    delete op;
    return s;
  }
  *out = op;
  return G4_OK;
}

g4_status g4_pages_extend(g4_pages* op, g4_stream stream, int32_t n_seq, const int32_t* d_slots, const int32_t* d_counts,
                          int32_t n_rows, int32_t* d_rows, int32_t* d_offsets, int32_t* d_new_lens) {
  if (!op || !d_slots || !d_counts || !d_offsets || !d_new_lens || !pages_count(op, n_seq) || n_rows < 0 || (n_rows && !d_rows))
    return G4_ERR_INVALID_ARG;
  // what a thread still reads, and what the call keeps up to date, are no outputs
  const long entries = (long)op->cfg.n_slots * op->cfg.max_pages;
  const struct { const int32_t* p; long n; } outs[3] = {{d_rows, n_rows}, {d_offsets, n_seq + 1L}, {d_new_lens, n_seq}};
  for (auto& o : outs)
    if (!pages_apart(o.p, o.n, op->p.table, entries) || !pages_apart(o.p, o.n, op->p.lens, op->cfg.n_slots)) return G4_ERR_INVALID_ARG;
  if (!pages_apart(d_rows, n_rows, d_offsets, n_seq + 1L) || !pages_apart(d_rows, n_rows, d_new_lens, n_seq) ||
      !pages_apart(d_offsets, n_seq + 1L, d_new_lens, n_seq) || !pages_apart(d_rows, n_rows, d_slots, n_seq) ||
      !pages_apart(d_rows, n_rows, d_counts, n_seq))
    return G4_ERR_INVALID_ARG;
  DEVICE_GUARD(op->device);
  PagesExtend a{op->p, d_slots, d_counts, n_seq, n_rows, d_rows, d_offsets, d_new_lens};
  launch(pages_extend_kernel, dim3(std::max(1, std::min(op->sms, cdiv(n_rows, 4 * kPagesThreads)))), dim3(kPagesThreads), 0,
         reinterpret_cast<cudaStream_t>(stream), a);
  CK(cudaGetLastError());
  return G4_OK;
}

g4_status g4_pages_share(g4_pages* op, g4_stream stream, int32_t n_seq, const int32_t* d_slots, int32_t source, int32_t n_pages) {
  if (!op || !d_slots || !pages_count(op, n_seq) || source < 0 || source >= op->cfg.n_slots || n_pages < 0 ||
      n_pages > op->cfg.max_pages)
    return G4_ERR_INVALID_ARG;
  DEVICE_GUARD(op->device);
  PagesShare a{op->p, d_slots, n_seq, source, n_pages};
  launch(pages_share_kernel, dim3(kPagesCluster), dim3(kPagesThreads), 0, reinterpret_cast<cudaStream_t>(stream), a);
  CK(cudaGetLastError());
  return G4_OK;
}

g4_status g4_pages_truncate(g4_pages* op, g4_stream stream, int32_t n_seq, const int32_t* d_slots, const int32_t* d_lens) {
  if (!op || !d_slots || !pages_count(op, n_seq)) return G4_ERR_INVALID_ARG;
  DEVICE_GUARD(op->device);
  PagesTruncate a{op->p, d_slots, d_lens, n_seq};
  launch(pages_truncate_kernel, dim3(kPagesCluster), dim3(kPagesThreads), 0, reinterpret_cast<cudaStream_t>(stream), a);
  CK(cudaGetLastError());
  return G4_OK;
}

g4_status g4_pages_store(g4_pages* op, g4_stream stream, int32_t n_rows, const int32_t* d_rows, int32_t num_kv_heads,
                         int32_t head_dim, const g4_kv4_tensor* k, const g4_kv4_tensor* v, void* k_pool, void* v_pool) {
  if (!op || !k || !v || !k_pool || !v_pool || n_rows < 0 || num_kv_heads < 1 || (n_rows && !d_rows)) return G4_ERR_INVALID_ARG;
  if (k->dtype != v->dtype || reinterpret_cast<uintptr_t>(k_pool) % 16 || reinterpret_cast<uintptr_t>(v_pool) % 16)
    return G4_ERR_INVALID_ARG;
  if ((k->dtype != G4_DT_BF16 && k->dtype != G4_DT_F16) || !paged_head_dim(head_dim) || (long)n_rows * num_kv_heads >= (1L << 31))
    return G4_ERR_UNSUPPORTED;
  if (!n_rows) return G4_OK;
  Paged16 pk, pv;
  if (!paged_tensor(k, n_rows, num_kv_heads, head_dim, false, &pk) || !paged_tensor(v, n_rows, num_kv_heads, head_dim, false, &pv))
    return G4_ERR_INVALID_ARG;
  DEVICE_GUARD(op->device);
  PagesStore a{};
  a.p = op->p;
  a.rows = d_rows;
  a.n_rows = n_rows;
  a.kvh = num_kv_heads;
  a.d8 = head_dim / 8;
  while ((1 << a.log_d8) < a.d8) ++a.log_d8;
  a.k = pk.p;
  a.v = pv.p;
  a.k_row = pk.row;
  a.k_head = pk.head;
  a.v_row = pv.row;
  a.v_head = pv.head;
  a.kp = static_cast<uint16_t*>(k_pool);
  a.vp = static_cast<uint16_t*>(v_pool);
  a.vec = pk.vec && pv.vec;
  const long pieces = (long)n_rows * num_kv_heads * a.d8, per = kPagesStoreThreads * kPagesStoreEach;
  launch(pages_store_kernel, dim3((unsigned)((pieces + per - 1) / per)), dim3(kPagesStoreThreads), 0,
         reinterpret_cast<cudaStream_t>(stream), a);
  CK(cudaGetLastError());
  return G4_OK;
}

g4_status g4_pages_get_device_error(g4_pages* op, g4_stream stream, int32_t* word_out) {
  if (!op) return G4_ERR_INVALID_ARG;
  return paged_error(op->device, op->p.err, stream, word_out);
}

int64_t g4_pages_bytes(const g4_pages* op) { return op ? (int64_t)op->mem.bytes : 0; }

void g4_pages_free(g4_pages* op) {
  if (!op) return;
  DeviceGuard dg(op->device);
  cudaDeviceSynchronize();
  cudaFree(op->mem.all);
  delete op;
}

}  // extern "C"
