// C entry points of the attention over 16-bit keys and values (include/g4.h, g4_attn_*).
#include <cmath>
#include <mutex>
#include <set>

#include "attn16_decode.cuh"
#include "paged_host.h"

using namespace g4;

struct g4_attn {
  g4_attn_config cfg{};
  int device = 0, sms = 0, smem_optin = 0;
  g4_paged_memory mem;
  int* err = nullptr;
  unsigned* ticket = nullptr;
  float *pre_o = nullptr, *tail_o = nullptr;      // parts of the prefix, of the rows behind it
  float2 *pre_ml = nullptr, *tail_ml = nullptr;
  int4* plan = nullptr;
};

namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled g_encode = nullptr;
std::mutex g_attn_mu;
std::set<int> g_attn_devices;  // devices whose kernels have their shared-memory limit set

#define ATT_DISPATCH(d, bf, ...)                                \
  {                                                             \
    auto att_run = [&](auto d_, auto bf_) {                     \
      constexpr int D = decltype(d_)::value;                    \
      constexpr bool BF = decltype(bf_)::value;                 \
      __VA_ARGS__;                                              \
    };                                                          \
    auto att_type = [&](auto d_) {                              \
      if (bf) att_run(d_, std::true_type{});                    \
      else att_run(d_, std::false_type{});                      \
    };                                                          \
    if (d == 64) att_type(std::integral_constant<int, 64>{});   \
    else if (d == 128) att_type(std::integral_constant<int, 128>{}); \
    else if (d == 256) att_type(std::integral_constant<int, 256>{}); \
    else att_type(std::integral_constant<int, 512>{});          \
  }

g4_status attn_init(int device, int optin) {
  std::lock_guard<std::mutex> lk(g_attn_mu);
  if (!g_encode) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r{};
    CK(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r));
    if (!f || r != cudaDriverEntryPointSuccess) return G4_ERR_CUDA;
    g_encode = reinterpret_cast<EncodeTiled>(f);
  }
  if (!g_attn_devices.insert(device).second) return G4_OK;
  for (int d : {64, 128, 256, 512})
    for (bool bf : {false, true})
      ATT_DISPATCH(d, bf, {
        set_max_dyn(att16_kernel<D, BF, false>, optin);
        set_max_dyn(att16_kernel<D, BF, true>, optin);
        set_max_dyn(att_tail_kernel<D, BF>, optin);
        carve_max(att_join_kernel<D, BF>);
      });
  cudaGetLastError();
  return G4_OK;
}

// Parts that the rows behind a prefix are cut into: two for each of the warps that take them (64 sequences of 550 to 1,100
// rows behind 16,384, eight heads of 128: one 76 us, two 69, four 72).
int attn_most(const g4_attn* op) {
  const int d = op->cfg.head_dim;
  return 2 * op->sms * (d <= 128 ? AttTail<128>::kWarps : d == 256 ? AttTail<256>::kWarps : AttTail<512>::kWarps);
}
int attn_group(const g4_attn* op) { return op->cfg.num_q_heads / op->cfg.num_kv_heads; }
int attn_tokens(const g4_attn* op) { return (op->cfg.head_dim <= 128 ? 2 : 1) * (kAttM / attn_group(op)); }  // of an item
int attn_half(const g4_attn* op) { return op->cfg.head_dim == 512 ? 2 : 1; }
// Parts that each item past `tiles` tiles of shared keys is cut into: one for each SM, or for every second where that leaves
// an SM 32 tiles at the most; the others begin with the rows behind the prefix meanwhile (64 sequences behind 16,384 rows,
// eight heads of 128: on 30% of the SMs 86 us, half 69, 70% 75, all 80).
int attn_splits(const g4_attn* op, int blocks, int tiles) {
  const int items = blocks * op->cfg.num_kv_heads * attn_half(op);
  const int sms = (long)items * tiles > 32L * op->sms / 2 ? op->sms : op->sms / 2;
  return std::max(1, std::min(tiles, sms / items));
}

// Whether the shared rows are attended to once for all, on the tensor cores, or by each sequence with its own rows, out of
// L2 after the first: a launch less, and short prefixes leave the tensor cores' kernel little but its start.  On their
// own up to 20 MB of rows in all, or 40 MB with up to 1,024 rows each.  Measured, microseconds once / on their own (300 own
// rows each): 8 x 2,048 rows, one head of 256 (17 MB) 14.8 / 15.1 and 3 fewer for the host; 8 x 512 13.3 / 12.1; 8 x 4,096
// (34 MB) 15.7 / 18.5; 8 x 1,024, eight heads of 128 (34 MB) 16.4 / 14.5; 64 x 256, one of 512 (34 MB) 27.4 / 18.9; 64 x
// 128 (34 MB) 20.2 / 12.6; 32 x 512 (67 MB) 20.1 / 23.3; 16 x 2,048 (134 MB) 19.1 / 29.5.  All with groups of up to eight heads;
// a wider group's rows are copied once for each eight of its heads, which is not counted.  (On their own, bf16 weights go into the
// products in two parts, once for all in one: g4_attn_shared tells the border.)
bool attn_once(const g4_attn* op, int n_seq, int rows) {
  const double bytes = 4.0 * n_seq * rows * op->cfg.num_kv_heads * op->cfg.head_dim;
  return bytes > (rows <= 1024 ? 40e6 : 20e6);
}

g4_status attn_create_impl(g4_attn* op, cudaStream_t st) {
  const g4_attn_config& f = op->cfg;
  const size_t group = attn_group(op), d = f.head_dim, rows = d <= 128 ? 2 * kAttM : kAttM;
  const size_t items = (size_t)cdiv(f.max_seqs, attn_tokens(op)) * f.num_kv_heads;
  const size_t parts = std::max<size_t>(items, op->sms) * rows;
  const size_t tails = ((size_t)attn_most(op) + (size_t)f.max_seqs * f.num_kv_heads * ((group + 7) / 8)) * 8;
  // (parts and the plan are written before they are read)
  return paged_alloc(&op->mem, 512, st, [&](auto& take) {
    take(&op->err, 1);
    take(&op->ticket, 2);
    take(&op->plan, (size_t)f.max_seqs);
    take(&op->pre_o, parts * d);
    take(&op->pre_ml, parts);
    take(&op->tail_o, tails * d);
    take(&op->tail_ml, tails);
  });
}

CUtensorMapDataType attn_type(const g4_attn* op) {
  return op->cfg.dtype == G4_DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}
// Rows of a packed tensor: `box` rows of one head and `slabs` times 64 numbers of them, 64 after 64.
bool attn_map_packed(const g4_attn* op, CUtensorMap* m, const Paged16& t, long rows, int box, int slabs) {
  const cuuint64_t dim[4] = {64, (cuuint64_t)op->cfg.num_kv_heads, (cuuint64_t)rows, (cuuint64_t)op->cfg.head_dim / 64};
  const long whole = (long)op->cfg.head_dim;  // (the stride of an axis of one is never taken)
  const cuuint64_t stride[3] = {(cuuint64_t)(dim[1] > 1 ? t.head : whole) * 2, (cuuint64_t)(rows > 1 ? t.row : whole) * 2, 128};
  const cuuint32_t boxes[4] = {64, 1, (cuuint32_t)box, (cuuint32_t)slabs}, step[4] = {1, 1, 1, 1};
  return g_encode(m, attn_type(op), 4, t.p, dim, stride, boxes, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Tokens of the queries: 64 numbers of all heads of a KV head, and as many tokens as a block has.
bool attn_map_queries(const g4_attn* op, CUtensorMap* m, const Paged16& t, long rows) {
  const int group = op->cfg.num_q_heads / op->cfg.num_kv_heads;
  const cuuint64_t dim[3] = {(cuuint64_t)op->cfg.head_dim, (cuuint64_t)op->cfg.num_q_heads, (cuuint64_t)rows};
  const long whole = (long)op->cfg.head_dim;
  const cuuint64_t stride[2] = {(cuuint64_t)(dim[1] > 1 ? t.head : whole) * 2, (cuuint64_t)(rows > 1 ? t.row : whole) * 2};
  const cuuint32_t boxes[3] = {64, (cuuint32_t)group, (cuuint32_t)(kAttM / group)}, step[3] = {1, 1, 1};
  return g_encode(m, attn_type(op), 3, t.p, dim, stride, boxes, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Whether the TMA can copy a tensor's rows.
bool attn_tma(const Paged16& t, long rows, long heads) {
  return reinterpret_cast<uintptr_t>(t.p) % 16 == 0 && (rows == 1 || (t.row % 8 == 0 && t.row > 0 && t.row < (1L << 38))) &&
         (heads == 1 || (t.head % 8 == 0 && t.head > 0 && t.head < (1L << 38)));
}
// Rows of a pool, all pages and heads one after the other.
bool attn_map_pool(const g4_attn* op, CUtensorMap* m, const void* pool, long rows, int box) {
  const cuuint64_t dim[2] = {(cuuint64_t)op->cfg.head_dim, (cuuint64_t)rows};
  const cuuint64_t stride[1] = {(cuuint64_t)op->cfg.head_dim * 2};
  const cuuint32_t boxes[2] = {64, (cuuint32_t)box}, step[2] = {1, 1};
  return g_encode(m, attn_type(op), 2, const_cast<void*>(pool), dim, stride, boxes, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool attn_scale(const g4_attn* op, float scale, float* out) {
  if (!(scale >= 0.f) || !std::isfinite(scale)) return false;
  const double x = (scale != 0.f ? (double)scale : 1.0 / std::sqrt((double)op->cfg.head_dim)) * 1.4426950408889634;
  *out = (float)std::min(x, 3.4028234663852886e38);
  return true;
}

}  // namespace

extern "C" {

g4_status g4_attn_create(int device, const g4_attn_config* cfg, g4_attn** out) {
  if (!out) return G4_ERR_INVALID_ARG;
  *out = nullptr;
  if (!cfg) return G4_ERR_INVALID_ARG;
  const g4_attn_config f = *cfg;
  if (f.num_q_heads < 1 || f.num_kv_heads < 1 || f.max_seqs < 1 || f.num_q_heads % f.num_kv_heads) return G4_ERR_INVALID_ARG;
  if (f.num_kv_heads > 64 || f.num_q_heads / f.num_kv_heads > 64 || f.max_seqs > kAttMaxSeqs || !paged_head_dim(f.head_dim) ||
      (f.dtype != G4_DT_BF16 && f.dtype != G4_DT_F16))
    return G4_ERR_UNSUPPORTED;
  DEVICE_GUARD(device);
  g4_attn* op = new (std::nothrow) g4_attn();
  if (!op) return G4_ERR_OOM;
  op->cfg = f;
  op->device = device;
  g4_status s = G4_ERR_CUDA;
  cudaStream_t st = nullptr;
  if (cuda_ok(cudaDeviceGetAttribute(&op->sms, cudaDevAttrMultiProcessorCount, device), "cudaDeviceGetAttribute") &&
      cuda_ok(cudaDeviceGetAttribute(&op->smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, device), "cudaDeviceGetAttribute") &&
      cuda_ok(cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking), "cudaStreamCreate")) {
    try {
      s = attn_init(device, op->smem_optin);
      if (s == G4_OK) s = attn_create_impl(op, st);
    } catch (...) {
      s = G4_ERR_OOM;
    }
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

g4_status g4_attn_prompt(g4_attn* op, g4_stream stream, int32_t n_seq, const int32_t* d_offsets, int32_t n_rows, float scale,
                         int32_t window, int32_t zero_rest, const g4_kv4_tensor* q, const g4_kv4_tensor* k,
                         const g4_kv4_tensor* v, const g4_kv4_tensor* out) {
  if (!op || !d_offsets || !q || !k || !v || !out || n_seq < 1 || n_seq > op->cfg.max_seqs || n_rows < 0 || window < 0)
    return G4_ERR_INVALID_ARG;
  const g4_attn_config& f = op->cfg;
  const int d = f.head_dim, group = f.num_q_heads / f.num_kv_heads;
  Att16Args a{};
  if (!attn_scale(op, scale, &a.scale)) return G4_ERR_INVALID_ARG;
  if (q->dtype != f.dtype || k->dtype != f.dtype || v->dtype != f.dtype || out->dtype != f.dtype) return G4_ERR_UNSUPPORTED;
  if (!n_rows) return G4_OK;
  Paged16 pq, pk, pv, po;
  if (!paged_tensor(q, n_rows, f.num_q_heads, d, false, &pq) || !paged_tensor(k, n_rows, f.num_kv_heads, d, false, &pk) ||
      !paged_tensor(v, n_rows, f.num_kv_heads, d, false, &pv) || !paged_tensor(out, n_rows, f.num_q_heads, d, true, &po) ||
      po.p == pq.p || po.p == pk.p || po.p == pv.p)
    return G4_ERR_INVALID_ARG;
  if ((long)n_rows * group >= (1L << 31)) return G4_ERR_UNSUPPORTED;
  if (!attn_tma(pq, n_rows, f.num_q_heads) || !attn_tma(pk, n_rows, f.num_kv_heads) || !attn_tma(pv, n_rows, f.num_kv_heads))
    return G4_ERR_UNSUPPORTED;
  DEVICE_GUARD(op->device);
  a.q = pq.p;
  a.out = po.p;
  a.k = pk.p;
  a.v = pv.p;
  a.q_row = pq.row;
  a.q_head = pq.head;
  a.o_row = po.row;
  a.o_head = po.head;
  a.k_row = pk.row;
  a.k_head = pk.head;
  a.v_row = pv.row;
  a.v_head = pv.head;
  a.o_vec = po.vec && reinterpret_cast<uintptr_t>(po.p) % 32 == 0 && po.row % 16 == 0 && po.head % 16 == 0 ? 2 : po.vec;
  a.group = group;
  a.kvh = f.num_kv_heads;
  a.tb = kAttM / group;
  a.err = op->err;
  a.offsets = d_offsets;
  a.n_seq = n_seq;
  a.n_rows = n_rows;
  a.window = window < n_rows ? window : 0;  // one that reaches every row is none
  a.ticket = op->ticket;
  a.zero_rest = zero_rest != 0;
  // every sequence's last item may be one that is not full
  const long blocks = n_rows / attn_tokens(op) + n_seq;
  const int ctas = (int)std::min<long>(op->sms, blocks * f.num_kv_heads * attn_half(op));
  bool ok = true;
  ATT_DISPATCH(d, f.dtype == G4_DT_BF16, {
    CUtensorMap qm;
    CUtensorMap km;
    CUtensorMap vm;
    ok = attn_map_queries(op, &qm, pq, n_rows) && attn_map_packed(op, &km, pk, n_rows, kAttN, Att16<D>::kStage / Att16<D>::kSlab) &&
         attn_map_packed(op, &vm, pv, n_rows, Att16<D>::kVRows, Att16<D>::DV / 64);
    if (ok)
      launch(att16_kernel<D, BF, false>, dim3(ctas), dim3(Att16<D>::kThreads), Att16<D>::kSmem, reinterpret_cast<cudaStream_t>(stream), a, qm, km, vm);
  });
  if (!ok) return G4_ERR_UNSUPPORTED;
  CK(cudaGetLastError());
  return G4_OK;
}

g4_status g4_attn_shared(g4_attn* op, g4_stream stream, const g4_pages* pages, int32_t n_seq, const int32_t* d_slots,
                         int32_t shared_pages, float scale, const void* k_pool, const void* v_pool, const g4_kv4_tensor* q,
                         const g4_kv4_tensor* out) {
  if (!op || !pages || !d_slots || !k_pool || !v_pool || !q || !out || n_seq < 1 || n_seq > op->cfg.max_seqs || shared_pages < 0 ||
      shared_pages > pages->cfg.max_pages || pages->device != op->device || reinterpret_cast<uintptr_t>(k_pool) % 16 ||
      reinterpret_cast<uintptr_t>(v_pool) % 16)
    return G4_ERR_INVALID_ARG;
  const g4_attn_config& f = op->cfg;
  const g4_pages_config& pf = pages->cfg;
  const int d = f.head_dim, group = f.num_q_heads / f.num_kv_heads;
  AttTailArgs t{};
  if (!attn_scale(op, scale, &t.scale)) return G4_ERR_INVALID_ARG;
  if (q->dtype != f.dtype || out->dtype != f.dtype) return G4_ERR_UNSUPPORTED;
  Paged16 pq, po;
  if (!paged_tensor(q, n_seq, f.num_q_heads, d, false, &pq) || !paged_tensor(out, n_seq, f.num_q_heads, d, true, &po) || po.p == pq.p)
    return G4_ERR_INVALID_ARG;
  if (!attn_tma(pq, n_seq, f.num_q_heads)) return G4_ERR_UNSUPPORTED;
  t.row_tiles = cdiv(group, 8);
  t.shared = shared_pages * pf.page_size;
  t.keys = attn_once(op, n_seq, t.shared) ? t.shared : 0;
  const long pool_rows = (long)pf.n_pages * f.num_kv_heads * pf.page_size;
  if (pool_rows >= (1L << 31) ||
      (double)n_seq * f.num_kv_heads * t.row_tiles * ((double)((long)pf.max_pages * pf.page_size - t.keys) / kAttBlock + 1) >= 2147483647.0)
    return G4_ERR_UNSUPPORTED;
  DEVICE_GUARD(op->device);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int blocks = cdiv(n_seq, attn_tokens(op)), tiles = cdiv(t.keys, kAttN);
  int splits = tiles ? attn_splits(op, blocks, tiles) : 0;
  const int tiles_per = splits ? cdiv(tiles, splits) : 0;
  if (splits) splits = cdiv(tiles, tiles_per);
  t.q = pq.p;
  t.q_row = pq.row;
  t.q_head = pq.head;
  t.kp = static_cast<const uint16_t*>(k_pool);
  t.vp = static_cast<const uint16_t*>(v_pool);
  t.out = po.p;
  t.o_row = po.row;
  t.o_head = po.head;
  t.o_vec = po.vec;
  t.n_seq = n_seq;
  t.group = group;
  t.kvh = f.num_kv_heads;
  t.table = pages->p.table;
  t.slots = d_slots;
  t.lens = pages->p.lens;
  t.n_slots = pf.n_slots;
  t.n_pages = pf.n_pages;
  t.log_page = pages->p.log_page;
  t.max_pages = pf.max_pages;
  t.part_o = op->tail_o;
  t.part_ml = op->tail_ml;
  t.plan = op->plan;
  t.most = attn_most(op);
  t.ticket = op->ticket;
  t.pre_o = op->pre_o;
  t.pre_ml = op->pre_ml;
  t.splits = splits;
  t.tb = kAttM / group;
  t.blocks = d <= 128 ? 2 : 1;
  t.err = op->err;
  bool ok = true;
  ATT_DISPATCH(d, f.dtype == G4_DT_BF16, {
    if (splits) {
      Att16Args a{};
      a.q = pq.p;
      a.q_row = pq.row;
      a.q_head = pq.head;
      a.group = group;
      a.kvh = f.num_kv_heads;
      a.tb = kAttM / group;
      a.scale = t.scale;
      a.err = op->err;
      a.n_seq = n_seq;
      a.table = t.table;
      a.slots = d_slots;
      a.lens = t.lens;
      a.n_slots = t.n_slots;
      a.n_pages = t.n_pages;
      a.log_page = t.log_page;
      a.max_pages = t.max_pages;
      a.keys = t.keys;
      a.splits = splits;
      a.tiles_per = tiles_per;
      a.part_o = op->pre_o;
      a.part_ml = op->pre_ml;
      CUtensorMap qm;
      CUtensorMap km;
      CUtensorMap vm;
      ok = attn_map_queries(op, &qm, pq, n_seq) && attn_map_pool(op, &km, k_pool, pool_rows, std::min(kAttN, pf.page_size)) &&
           attn_map_pool(op, &vm, v_pool, pool_rows, std::min(Att16<D>::kVRows, pf.page_size));
      const int items = blocks * f.num_kv_heads * splits * Att16<D>::HV;
      if (ok)
        launch(att16_kernel<D, BF, true>, dim3(std::min(items, op->sms)), dim3(Att16<D>::kThreads), Att16<D>::kSmem, st, a, qm, km, vm);
    }
    if (ok) {
      launch(att_tail_kernel<D, BF>, dim3(op->sms), dim3(32 * AttTail<D>::kWarps), AttTail<D>::smem(n_seq), st, t);
      launch(att_join_kernel<D, BF>, dim3(n_seq * f.num_q_heads), dim3(32 * kAttJoinWarps), 0, st, t);
    }
  });
  if (!ok) return G4_ERR_UNSUPPORTED;
  CK(cudaGetLastError());
  return G4_OK;
}

g4_status g4_attn_get_device_error(g4_attn* op, g4_stream stream, int32_t* word_out) {
  if (!op) return G4_ERR_INVALID_ARG;
  return paged_error(op->device, op->err, stream, word_out);
}

int64_t g4_attn_bytes(const g4_attn* op) { return op ? (int64_t)op->mem.bytes : 0; }

void g4_attn_free(g4_attn* op) {
  if (!op) return;
  DeviceGuard dg(op->device);
  cudaDeviceSynchronize();
  cudaFree(op->mem.all);
  delete op;
}

}  // extern "C"
