// C entry points of the 4-bit KV cache (include/g4.h, g4_kv4_*): argument checks, the handle
// with its cache and workspace, and the launches of kv4.cuh, kv4_attend.cuh and kv4_block.cuh.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <mutex>
#include <new>
#include <set>
#include <vector>

#include "host.h"
#include "kv4.cuh"
#include "kv4_attend.cuh"
#include "kv4_block.cuh"
#include "kv4_host.h"

using namespace g4;

struct g4_kv4 {
  g4_kv4_config cfg{};
  int device = 0;
  Kv4Cache c{};
  std::vector<void*> allocs;
  size_t bytes = 0;
  int fail_at = 0, n_allocs = 0;  // allocation-failure injection (G4_FAIL_ALLOC_AT), as in g4_create
  Kv4Work work;
  int *holes = nullptr, *movers = nullptr;    // evict: [n_slots][kvh][capacity / 2]
  int* n_moves = nullptr;                     // [n_slots][kvh]
};

namespace {

template <class T>
g4_status kv4_alloc(g4_kv4* op, T** p, size_t count, cudaStream_t st) {
  void* q = nullptr;
  const size_t n = std::max<size_t>(count, 1) * sizeof(T);
  if (op->fail_at > 0 && ++op->n_allocs == op->fail_at) return G4_ERR_OOM;  // injected
  const cudaError_t e = cudaMalloc(&q, n);
  if (e != cudaSuccess) {
    cuda_ok(e, "cudaMalloc");
    cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? G4_ERR_OOM : G4_ERR_CUDA;
  }
  op->allocs.push_back(q);
  op->bytes += n;
  *p = static_cast<T*>(q);
  CK(cudaMemsetAsync(q, 0, n, st));
  return G4_OK;
}

int log2i(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

// Tensor argument -> kernel form.  [n][rows][heads][d]; false when it is malformed.
bool kv4_dense(const g4_kv4_tensor* t, long n, long rows, long heads, int d, bool written, Kv4Dense* out) {
  *out = Kv4Dense{};
  if (!t) return true;
  if (!t->data || t->dtype < G4_DT_F32 || t->dtype > G4_DT_F16) return false;
  const long es = t->dtype == G4_DT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(t->data) % es) return false;
  struct { long stride, size; } ax[3] = {{(long)t->seq_stride, n}, {(long)t->row_stride, rows}, {(long)t->head_stride, heads}};
  const long most = 1L << 46;  // keeps every offset far inside 64 bits
  for (auto& x : ax)
    if (x.stride < 0 || x.stride > most / std::max(x.size, 1L)) return false;
  if (written) {  // no element twice: each stride steps over all that smaller strides reach
    std::sort(ax, ax + 3, [](auto& x, auto& y) { return x.stride < y.stride; });
    long extent = d;
    for (auto& x : ax) {
      if (x.size <= 1) continue;
      if (x.stride < extent) return false;
      extent += x.stride * (x.size - 1);
    }
  }
  out->p = t->data;
  out->seq = t->seq_stride;
  out->row = t->row_stride;
  out->head = t->head_stride;
  out->dtype = t->dtype;
  auto aligned = [&](long bytes) {
    const long n = bytes / es;
    return reinterpret_cast<uintptr_t>(t->data) % bytes == 0 && t->seq_stride % n == 0 && t->row_stride % n == 0 &&
           t->head_stride % n == 0;
  };
  out->vec = aligned(32) ? 2 : aligned(16) ? 1 : 0;
  return true;
}

bool kv4_count(const g4_kv4* op, int n_seq) { return n_seq >= 1 && n_seq <= op->cfg.n_slots; }

// A kernel for the handle's head dim.
#define KV4_DISPATCH(d, ...)                         \
  switch (d) {                                       \
    case 64: { constexpr int D = 64; __VA_ARGS__; break; }    \
    case 128: { constexpr int D = 128; __VA_ARGS__; break; }  \
    case 256: { constexpr int D = 256; __VA_ARGS__; break; }  \
    default: { constexpr int D = 512; __VA_ARGS__; break; }   \
  }

#define KV4_DISPATCH_TYPE(dt, ...)                                       \
  switch (dt) {                                                          \
    case G4_DT_F32: { constexpr int DT = G4_DT_F32; __VA_ARGS__; break; }   \
    case G4_DT_F16: { constexpr int DT = G4_DT_F16; __VA_ARGS__; break; }   \
    default: { constexpr int DT = G4_DT_BF16; __VA_ARGS__; break; }         \
  }

std::mutex g_kv4_mu;
std::set<int> g_kv4_devices;  // devices whose kernels have their shared-memory limit set
template <int D, int DT>
void kv4_attrs(int optin) {
  set_max_dyn(kv4_attend_kernel<D, DT>, optin);
  set_max_dyn(kv4_gain_kernel<D, DT>, optin);
  set_max_dyn(kv4_finish_kernel<D, DT>, optin);
}
template <int D>
void kv4_attrs_block(int optin) {
  set_max_dyn(kv4_block_kernel<D, false>, optin);
  set_max_dyn(kv4_block_kernel<D, true>, optin);
  carve_max(kv4_block_join_kernel<D>);
}
template <int D>
void kv4_attrs_d(int optin) {
  kv4_attrs<D, G4_DT_F32>(optin);
  kv4_attrs<D, G4_DT_BF16>(optin);
  kv4_attrs<D, G4_DT_F16>(optin);
  carve_max(kv4_append_kernel<D>);
  carve_max(kv4_append_blocks_kernel<D>);
  carve_max(kv4_step_kernel<D>);
  carve_max(kv4_read_blocks_kernel<D>);
  carve_max(kv4_read_kernel<D>);
  carve_max(kv4_move_kernel<D>);
}
int kv4_most_moves(const g4_kv4* op) { return std::max(1, op->cfg.capacity / 2); }
int kv4_row_tiles(const g4_kv4* op, int q_len) { return cdiv(q_len * (op->cfg.num_q_heads / op->cfg.num_kv_heads), 8); }

// Blocks of query tokens on the 5th-generation tensor cores (kv4_block.cuh).
bool kv4_block_path(const g4_kv4* op, int q_len, int dtype) {
  return dtype == G4_DT_BF16 && op->cfg.head_dim <= 256 && q_len * (op->cfg.num_q_heads / op->cfg.num_kv_heads) > kv4_block_rows(op->cfg.head_dim);
}
// Shared memory of kv4_plan in a kernel that has no other use for the table's.
size_t kv4_plan_smem(const Kv4AttendArgs& a) { return (size_t)a.n_seq * 20 + 16 + (a.accumulate ? (size_t)a.c.n_slots * 4 : 0); }
template <int D>
void kv4_launch_block(const Kv4Work& op, Kv4AttendArgs a, cudaStream_t st) {
  const int rows = a.q_len * a.group;
  a.row_tiles = cdiv(rows, kKv4M);
  a.lse_rows = a.row_tiles * kKv4M;
  a.join_inside = 0;
  launch(kv4_block_kernel<D, false>, dim3(op.sms), dim3(kKv4BlockThreads), Kv4Blk<D, false>::smem(a.n_seq), st, a);
  launch(kv4_block_join_kernel<D>, dim3(a.n_seq * a.c.kvh * a.row_tiles, D / 16), dim3(kKv4M), kv4_plan_smem(a),
         st, a, op.sms);
  if (!a.accumulate) return;
  a.row_tiles = 1;  // the account cuts the keys alone into spans
  launch(kv4_block_kernel<D, true>, dim3(op.sms), dim3(kKv4BlockThreads), Kv4Blk<D, true>::smem(a.n_seq), st, a);
}

// The softmax scale in the base-2 exponentials' units.  Narrow codes stand for 2^-64 of their values
// (Kv4Scale), which the kernels make up for by 2^64 times the scale; where that passes fp32's range
// the codes are decoded the plain way.
void kv4_set_scale(Kv4AttendArgs& a, double scale) {
  a.scale = (float)std::min(scale * 1.4426950408889634, (double)FLT_MAX);
  a.plain = !std::isfinite(a.scale * kKv4Up);
}

void kv4_use(const Kv4Work& w, Kv4AttendArgs& a) {
  a.lse = w.lse;
  a.lse_rows = a.row_tiles * 8;
  a.part_o = w.part_o;
  a.part_ml = w.part_ml;
  a.tickets = w.tickets;
}

template <int D, int DT>
void kv4_launch_attend(const Kv4Work& op, Kv4AttendArgs& a, cudaStream_t st) {
  using C = Kv4Att<D, DT>;
  const int ctas = op.sms * C::kMinCtas;
  // the ring takes what shared memory the CTAs of an SM leave each other (1 KB each is the system's)
  const int room = (op.smem_optin + 1024) / C::kMinCtas - 1024 - (int)C::smem(0, a.n_seq);
  a.stages = kv4_ring_stages(room, C::kTile, C::kSets);
  const int items = a.n_seq * a.c.kvh * a.row_tiles;
  // Parts of shared items are joined by the last CTA to finish one (a launch less), or by a second
  // launch with CTAs enough for the parts of long items.  Inside: with more items than CTAs, where the
  // second launch would have a CTA or more for each, and with few tiles a slot.  Measured, microseconds
  // inside / second launch.  One sequence of 200 rows, D = 256: 11.0 / 11.6, D = 512 and 450 rows: 16.5 /
  // 19.3; 512 sequences of 640, 256: 53.5 / 57.4, 1,024: 88.2 / 115.5; 1,024 of 300 rows, eight heads of
  // 64: 116 / 167.  64 sequences of 640, 256: 20.5 / 16.6; 64 of 3,000, 64: 18.5 / 14.4; eight of 8,000,
  // eight heads of 128: 30.7 / 26.8; 64 of those (512 items, 456 CTAs): 109.2 / 108.6.
  a.join_inside = items > ctas || cdiv(a.c.capacity, C::kKeys) <= kKv4Join;
  launch(kv4_attend_kernel<D, DT>, dim3(ctas), dim3(C::kThreads), C::smem(a.stages, a.n_seq), st, a);
  const int join_ctas = a.join_inside ? 0 : std::max(1, D * 2 / kKv4FinishThreads);
  const bool one = a.row_tiles == 1;  // the account of a single row tile rides along with the join
  const int gain_ctas = one && a.accumulate ? std::max(1, std::min(cdiv(a.c.capacity, 4 * kKv4Block), cdiv(8 * op.sms, items))) : 0;
  if (join_ctas + gain_ctas)
    launch(kv4_finish_kernel<D, DT>, dim3(items, join_ctas + gain_ctas), dim3(kKv4FinishThreads),
           kv4_plan_smem(a) + C::kQBytes, st, a, ctas, join_ctas);
  if (a.accumulate && !one)
    launch(kv4_gain_kernel<D, DT>, dim3(std::max(1, std::min(cdiv(a.c.capacity, 64), 8 * op.sms / a.n_seq)), a.n_seq, a.c.kvh),
           dim3(32 * kKv4GainWarps), C::kQBytes, st, a);
}

// Whether rows go by whole blocks (a warp each) or by octets (a thread each): by blocks from
// per_sm blocks per SM on, where the octets' scattered accesses cost more than the blocks' longer
// chains.  Measured (D = 256, fp32; microseconds by blocks / by octets): append of 104 blocks 9.3 /
// 5.2, 320: 10.0 / 9.3, 416: 10.3 / 10.4, 1,280: 16.8 / 23.2, 4,096: 36 / 66; read of 32: 3.6 / 3.1,
// 104: 3.6 / 3.6, 320: 4.2 / 5.7, 4,096: 15 / 32.
bool kv4_by_blocks(const g4_kv4* op, int n_seq, int n_rows, int per_sm) {
  return n_rows >= kKv4Block && (long)n_seq * op->cfg.num_kv_heads * cdiv(n_rows, kKv4Block) >= (long)per_sm * op->work.sms;
}
// Whole-block kernels: every block that n_rows rows from any row on can touch.
dim3 kv4_block_grid(const g4_kv4* op, int n_seq, int n_rows) {
  const long units = ((long)(n_rows + 2 * kKv4Block - 2) / kKv4Block) * op->cfg.num_kv_heads;
  return dim3((unsigned)((units + kKv4BlockWarps - 1) / kKv4BlockWarps), n_seq, 2);
}
dim3 kv4_row_grid(const g4_kv4* op, int n_seq, int n_rows) {
  const long threads = (long)n_rows * op->cfg.num_kv_heads * (op->cfg.head_dim / 8);
  return dim3((unsigned)((threads + kKv4RowThreads - 1) / kKv4RowThreads), n_seq);
}

g4_status kv4_create_impl(g4_kv4* op, const int32_t* d_page_table, cudaStream_t st) {
  const g4_kv4_config& f = op->cfg;
  Kv4Cache& c = op->c;
  c.n_slots = f.n_slots;
  c.capacity = f.capacity;
  c.kvh = f.num_kv_heads;
  c.d = f.head_dim;
  size_t blocks;
  if (f.page_size) {
    c.table = d_page_table;
    c.bpp = f.page_size / kKv4Block;
    c.log_bpp = log2i(c.bpp);
    c.max_pages = cdiv(f.capacity, f.page_size);
    c.n_pages = f.n_pages;
    blocks = (size_t)f.n_pages * c.kvh * c.bpp;
  } else {
    c.bpp = cdiv(f.capacity, kKv4Block);
    blocks = (size_t)f.n_slots * c.kvh * c.bpp;
  }
  TRY(kv4_alloc(op, &c.data, blocks * 18 * f.head_dim, st));
  TRY(kv4_alloc(op, &c.wide, 1, st));
  TRY(kv4_alloc(op, &c.err, 1, st));
  const bool blocks_too = kv4_block_path(op, f.max_q_len, G4_DT_BF16);
  const int group = f.num_q_heads / f.num_kv_heads;
  const size_t lse = kv4_work_lse(f.n_slots, c.kvh, group, f.max_q_len), lse_blocks = (size_t)f.n_slots * c.kvh * cdiv(f.max_q_len * group, kKv4M) * kKv4M;
  TRY(kv4_alloc(op, &op->work.lse, blocks_too ? std::max(lse, lse_blocks) : lse, st));
  // two partial items of every CTA, of 8 query rows each, or 128
  const size_t part_rows = std::max(kv4_work_part_rows(op->work.sms), blocks_too ? (size_t)2 * op->work.sms * kKv4M : 0);
  TRY(kv4_alloc(op, &op->work.part_o, part_rows * f.head_dim / 4, st));
  TRY(kv4_alloc(op, &op->work.part_ml, part_rows, st));
  TRY(kv4_alloc(op, &op->work.tickets, kv4_work_tickets(f.n_slots, c.kvh, group, f.max_q_len), st));
  if (f.track) {
    TRY(kv4_alloc(op, &c.pos, blocks * kKv4Block, st));
    TRY(kv4_alloc(op, &c.weight, blocks * kKv4Block, st));
    TRY(kv4_alloc(op, &c.base, (size_t)f.n_slots * c.kvh, st));
    // at most half of a slot's rows move: a move takes an evicted row below the budget and a
    // kept one beyond it
    TRY(kv4_alloc(op, &op->holes, (size_t)f.n_slots * c.kvh * kv4_most_moves(op), st));
    TRY(kv4_alloc(op, &op->movers, (size_t)f.n_slots * c.kvh * kv4_most_moves(op), st));
    TRY(kv4_alloc(op, &op->n_moves, (size_t)f.n_slots * c.kvh, st));
  }
  return G4_OK;
}

}  // namespace

// ------------------------------------------------------------------ for the decode step
namespace g4 {

void kv4_init(int device, int smem_optin) {
  std::lock_guard<std::mutex> lk(g_kv4_mu);
  if (!g_kv4_devices.insert(device).second) return;
  kv4_attrs_d<64>(smem_optin);
  kv4_attrs_d<128>(smem_optin);
  kv4_attrs_d<256>(smem_optin);
  kv4_attrs_d<512>(smem_optin);
  kv4_attrs_block<64>(smem_optin);
  kv4_attrs_block<128>(smem_optin);
  kv4_attrs_block<256>(smem_optin);
  carve_max(kv4_account_kernel);
  set_max_dyn(kv4_select_kernel, smem_optin);
  cudaGetLastError();
}

size_t kv4_work_lse(int n_seq, int kvh, int group, int q_len) { return (size_t)n_seq * kvh * cdiv(q_len * group, 8) * 8; }
size_t kv4_work_part_rows(int sms) { return (size_t)2 * sms * 8 * kKv4MaxCtas; }
size_t kv4_work_tickets(int n_seq, int kvh, int group, int q_len) { return (size_t)n_seq * kvh * cdiv(q_len * group, 8); }
size_t kv4_cache_bytes(size_t blocks, int kvh, int head_dim) { return blocks * kvh * 18 * head_dim; }

void kv4_step_rows(const Kv4Cache& c, const Kv4Step& a, int n, cudaStream_t st) {
  KV4_DISPATCH(c.d, launch(kv4_step_kernel<D>, dim3(a.nq + (a.own ? 1 : 0), n), dim3(32), 0, st, c, a));
}

void kv4_step_attend(const Kv4Cache& c, const Kv4Work& w, int n, const int* slots, const int* lens, int nq, float scale,
                     int window, float* q, float* out, int out_stride, cudaStream_t st) {
  Kv4AttendArgs a{};
  a.c = c;
  a.slots = slots;
  a.lens = lens;
  a.n_seq = n;
  a.q_len = 1;
  a.heads = a.group = nq;
  a.row_tiles = cdiv(nq, 8);
  kv4_set_scale(a, scale);
  a.window = window;
  a.q = Kv4Dense{q, (long)nq * c.d, (long)nq * c.d, c.d, G4_DT_F32, 2};
  a.out = Kv4Dense{out, out_stride, out_stride, c.d, G4_DT_F32, out_stride % 8 == 0 ? 2 : 0};
  kv4_use(w, a);
  KV4_DISPATCH(c.d, (kv4_launch_attend<D, G4_DT_F32>(w, a, st)));
}

}  // namespace g4

extern "C" {

g4_status g4_kv4_create(int device, const g4_kv4_config* cfg, const int32_t* d_page_table, g4_kv4** out) {
  if (!out) return G4_ERR_INVALID_ARG;
  *out = nullptr;
  if (!cfg) return G4_ERR_INVALID_ARG;
  const g4_kv4_config f = *cfg;
  if (f.n_slots < 1 || f.capacity < 1 || f.num_q_heads < 1 || f.num_kv_heads < 1 || f.max_q_len < 1 || f.page_size < 0 ||
      f.track < 0 || f.track > 1)
    return G4_ERR_INVALID_ARG;
  if (f.num_q_heads % f.num_kv_heads) return G4_ERR_INVALID_ARG;
  if (f.page_size ? (!d_page_table || f.n_pages < 1) : (d_page_table != nullptr)) return G4_ERR_INVALID_ARG;
  if (f.n_slots > kKv4MaxSlots || f.capacity > (1 << 20) || f.num_kv_heads > 64 || f.max_q_len > 64 ||
      f.num_q_heads / f.num_kv_heads > 64)
    return G4_ERR_UNSUPPORTED;
  if (f.head_dim != 64 && f.head_dim != 128 && f.head_dim != 256 && f.head_dim != 512) return G4_ERR_UNSUPPORTED;
  if (f.page_size && (f.page_size < kKv4Block || f.page_size > (1 << 20) || (f.page_size & (f.page_size - 1)) || f.n_pages > (1 << 26)))
    return G4_ERR_UNSUPPORTED;
  DEVICE_GUARD(device);
  g4_kv4* op = new (std::nothrow) g4_kv4();
  if (!op) return G4_ERR_OOM;
  op->cfg = f;
  op->device = device;
  if (const char* fa = getenv("G4_FAIL_ALLOC_AT")) op->fail_at = atoi(fa);
  g4_status s = G4_ERR_CUDA;
  cudaStream_t st = nullptr;
  if (cuda_ok(cudaDeviceGetAttribute(&op->work.sms, cudaDevAttrMultiProcessorCount, device), "cudaDeviceGetAttribute") &&
      cuda_ok(cudaDeviceGetAttribute(&op->work.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, device), "cudaDeviceGetAttribute") &&
      cuda_ok(cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking), "cudaStreamCreate")) {
    try {
      op->allocs.reserve(32);  // so that no allocation is lost for want of a place to note it
      kv4_init(device, op->work.smem_optin);
      s = kv4_create_impl(op, d_page_table, st);
    } catch (...) {
      s = G4_ERR_OOM;
    }
    if (!cuda_ok(cudaStreamSynchronize(st), "cudaStreamSynchronize") && s == G4_OK) s = G4_ERR_CUDA;
    cudaStreamDestroy(st);
  }
  if (s != G4_OK) {
    for (void* p : op->allocs) cudaFree(p);
    delete op;
    return s;
  }
  *out = op;
  return G4_OK;
}

g4_status g4_kv4_append(g4_kv4* op, g4_stream stream, int32_t n_seq, const int32_t* d_slots, const int32_t* d_start,
                        const int32_t* d_counts, int32_t n_rows, const g4_kv4_tensor* k, const g4_kv4_tensor* v,
                        const int32_t* d_positions, const float* d_weights) {
  if (!op || !d_slots || !d_start || !k || !v || !kv4_count(op, n_seq) || n_rows < 1 || n_rows > op->cfg.capacity)
    return G4_ERR_INVALID_ARG;
  Kv4RowArgs a{};
  if (!kv4_dense(k, n_seq, n_rows, op->c.kvh, op->c.d, false, &a.k) ||
      !kv4_dense(v, n_seq, n_rows, op->c.kvh, op->c.d, false, &a.v))
    return G4_ERR_INVALID_ARG;
  if (!op->cfg.track && (d_positions || d_weights)) return G4_ERR_UNSUPPORTED;
  DEVICE_GUARD(op->device);
  a.c = op->c;
  a.slots = d_slots;
  a.start = d_start;
  a.counts = d_counts;
  a.n_rows = n_rows;
  a.positions = d_positions;
  a.weights = d_weights;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool blocks = kv4_by_blocks(op, n_seq, n_rows, 3);
  dim3 grid = blocks ? kv4_block_grid(op, n_seq, n_rows) : kv4_row_grid(op, n_seq, n_rows);
  grid.x += op->cfg.track;  // kv4_set_bases
  if (blocks) {
    KV4_DISPATCH(op->c.d, launch(kv4_append_blocks_kernel<D>, grid, dim3(32 * kKv4BlockWarps), 0, st, a));
  } else {
    KV4_DISPATCH(op->c.d, launch(kv4_append_kernel<D>, grid, dim3(kKv4RowThreads), 0, st, a));
  }
  CK(cudaGetLastError());
  return G4_OK;
}

g4_status g4_kv4_read(g4_kv4* op, g4_stream stream, int32_t n_seq, const int32_t* d_slots, const int32_t* d_start,
                      const int32_t* d_counts, int32_t n_rows, int32_t zero_rest, const g4_kv4_tensor* k,
                      const g4_kv4_tensor* v) {
  if (!op || !d_slots || !d_start || (!k && !v) || !kv4_count(op, n_seq) || n_rows < 1 || n_rows > op->cfg.capacity)
    return G4_ERR_INVALID_ARG;
  Kv4RowArgs a{};
  if (!kv4_dense(k, n_seq, n_rows, op->c.kvh, op->c.d, true, &a.k) ||
      !kv4_dense(v, n_seq, n_rows, op->c.kvh, op->c.d, true, &a.v))
    return G4_ERR_INVALID_ARG;
  DEVICE_GUARD(op->device);
  a.c = op->c;
  a.slots = d_slots;
  a.start = d_start;
  a.counts = d_counts;
  a.n_rows = n_rows;
  a.zero_rest = zero_rest != 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (kv4_by_blocks(op, n_seq, n_rows, 1)) {
    KV4_DISPATCH(op->c.d, launch(kv4_read_blocks_kernel<D>, kv4_block_grid(op, n_seq, n_rows), dim3(32 * kKv4BlockWarps), 0, st, a));
  } else {
    KV4_DISPATCH(op->c.d, launch(kv4_read_kernel<D>, kv4_row_grid(op, n_seq, n_rows), dim3(kKv4RowThreads), 0, st, a));
  }
  CK(cudaGetLastError());
  return G4_OK;
}

g4_status g4_kv4_account(g4_kv4* op, g4_stream stream, int32_t n_seq, const int32_t* d_slots, const int32_t* d_start,
                         const int32_t* d_counts, int32_t n_rows, int32_t zero_rest, int32_t* d_positions,
                         float* d_weights) {
  if (!op || !d_slots || !d_start || (!d_positions && !d_weights) || !kv4_count(op, n_seq) || n_rows < 1 ||
      n_rows > op->cfg.capacity)
    return G4_ERR_INVALID_ARG;
  if (!op->cfg.track) return G4_ERR_UNSUPPORTED;
  DEVICE_GUARD(op->device);
  Kv4RowArgs a{};
  a.c = op->c;
  a.slots = d_slots;
  a.start = d_start;
  a.counts = d_counts;
  a.n_rows = n_rows;
  a.zero_rest = zero_rest != 0;
  a.positions_out = d_positions;
  a.weights_out = d_weights;
  launch(kv4_account_kernel, dim3(cdiv(n_rows, kKv4RowThreads), n_seq, op->c.kvh), dim3(kKv4RowThreads), 0,
         reinterpret_cast<cudaStream_t>(stream), a);
  CK(cudaGetLastError());
  return G4_OK;
}

g4_status g4_kv4_attend(g4_kv4* op, g4_stream stream, int32_t n_seq, const int32_t* d_slots, const int32_t* d_lens,
                        int32_t q_len, const int32_t* d_q_lens, float scale, int32_t window, int32_t accumulate,
                        int32_t zero_rest, const g4_kv4_tensor* q, const g4_kv4_tensor* out) {
  if (!op || !d_slots || !d_lens || !q || !out || !kv4_count(op, n_seq) || q_len < 1 || q_len > op->cfg.max_q_len ||
      window < 0 || !(scale >= 0.f) || !std::isfinite(scale) || q->dtype != out->dtype || q->data == out->data)
    return G4_ERR_INVALID_ARG;
  Kv4AttendArgs a{};
  if (!kv4_dense(q, n_seq, q_len, op->cfg.num_q_heads, op->c.d, false, &a.q) ||
      !kv4_dense(out, n_seq, q_len, op->cfg.num_q_heads, op->c.d, true, &a.out))
    return G4_ERR_INVALID_ARG;
  if ((accumulate && !op->cfg.track) || (window && op->cfg.track)) return G4_ERR_UNSUPPORTED;
  // the spans count (key tile, eight query rows) pairs in 32 bits
  if ((double)n_seq * op->c.kvh * kv4_row_tiles(op, q_len) * cdiv(op->cfg.capacity, 64) >= 2147483647.0) return G4_ERR_UNSUPPORTED;
  DEVICE_GUARD(op->device);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  a.c = op->c;
  a.slots = d_slots;
  a.lens = d_lens;
  a.q_lens = d_q_lens;
  a.n_seq = n_seq;
  a.q_len = q_len;
  a.heads = op->cfg.num_q_heads;
  a.group = a.heads / op->c.kvh;
  a.row_tiles = kv4_row_tiles(op, q_len);
  kv4_set_scale(a, scale != 0.f ? (double)scale : 1.0 / std::sqrt((double)op->c.d));
  a.window = window < op->cfg.capacity ? window : 0;  // one that reaches every row is none
  a.accumulate = accumulate != 0;
  a.zero_rest = zero_rest != 0;
  kv4_use(op->work, a);
  // (a few hundred sequences' spans no longer fit beside the operands of a 256-wide head)
  if (kv4_block_path(op, q_len, q->dtype) && (int)Kv4Blk<256, false>::smem(n_seq) <= op->work.smem_optin) {
    switch (op->c.d) {
      case 64: kv4_launch_block<64>(op->work, a, st); break;
      case 128: kv4_launch_block<128>(op->work, a, st); break;
      default: kv4_launch_block<256>(op->work, a, st); break;
    }
  } else {
    KV4_DISPATCH(op->c.d, KV4_DISPATCH_TYPE(q->dtype, (kv4_launch_attend<D, DT>(op->work, a, st))));
  }
  CK(cudaGetLastError());
  return G4_OK;
}

g4_status g4_kv4_evict(g4_kv4* op, g4_stream stream, int32_t n_seq, const int32_t* d_slots, const int32_t* d_lens,
                       int32_t budget, int32_t recent, int32_t* d_new_lens) {
  if (!op || !d_slots || !d_lens || !d_new_lens || d_new_lens == d_lens || !kv4_count(op, n_seq) || budget < 1 ||
      budget > op->cfg.capacity || recent < 0 || recent > budget)
    return G4_ERR_INVALID_ARG;
  if (!op->cfg.track) return G4_ERR_UNSUPPORTED;
  DEVICE_GUARD(op->device);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Kv4EvictArgs a{};
  a.c = op->c;
  a.slots = d_slots;
  a.lens = d_lens;
  a.budget = budget;
  a.recent = recent;
  a.new_lens = d_new_lens;
  a.holes = op->holes;
  a.movers = op->movers;
  a.n_moves = op->n_moves;
  a.most = kv4_most_moves(op);
  a.smem_rows = std::min(op->cfg.capacity, (op->work.smem_optin - 4096) / 4);
  launch(kv4_select_kernel, dim3(n_seq, op->c.kvh), dim3(kKv4EvictThreads), (size_t)a.smem_rows * 4, st, a);
  const int per = kKv4RowThreads / (op->c.d / 8);  // moves of a CTA at a time
  const int most = std::min(budget, op->cfg.capacity - budget);
  if (most > 0)
    KV4_DISPATCH(op->c.d, launch(kv4_move_kernel<D>, dim3(std::min(cdiv(most, per), std::max(1, cdiv(8 * op->work.sms, n_seq * op->c.kvh))), n_seq, op->c.kvh),
                                 dim3(kKv4RowThreads), 0, st, a));
  CK(cudaGetLastError());
  return G4_OK;
}

g4_status g4_kv4_get_device_error(g4_kv4* op, g4_stream stream, int32_t* word_out) {
  if (!op) return G4_ERR_INVALID_ARG;
  DEVICE_GUARD(op->device);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int w = 0;
  CK(cudaMemcpyAsync(&w, op->c.err, sizeof(int), cudaMemcpyDeviceToHost, st));
  CK(cudaMemsetAsync(op->c.err, 0, sizeof(int), st));
  CK(cudaStreamSynchronize(st));
  if (word_out) *word_out = w;
  if (w & G4_DEV_TIMEOUT) return G4_ERR_TIMEOUT;
  return w ? G4_ERR_DEVICE_CHECK : G4_OK;
}

int64_t g4_kv4_bytes(const g4_kv4* op) { return op ? (int64_t)op->bytes : 0; }

void g4_kv4_free(g4_kv4* op) {
  if (!op) return;
  DeviceGuard dg(op->device);
  cudaDeviceSynchronize();
  for (void* p : op->allocs) cudaFree(p);
  delete op;
}

}  // extern "C"
