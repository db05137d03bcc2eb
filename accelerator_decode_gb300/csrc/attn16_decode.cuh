// Attention of one token per sequence over a batch's rows behind their shared prefix, and the join of
// those parts with the prefix's (attn16.cuh).
//
// HBM bounds it: with up to eight query heads per KV head every row is copied once, with more once for each eight of
// them (out of L2 after the first, where they come at about the same time).  A block is 16 rows of one KV head, which lie one after the
// other in one page: a warp copies blocks into a ring of its own by two bulk copies each.  With the rows
// as the matrix instructions' 16-row operand and up to eight query heads as their columns,
//   S^T (16 keys x 8) = K Q^T     O^T (16 numbers x 8) += V^T P^T,
// 16-byte loads from the ring are the operands as they come: a permutation of the head dim that keys and
// queries share, and pairs of values' rows interleaved by a byte permutation.  O^T takes D / 4
// registers a lane, the queries D / 8.
// Every item (sequence, KV head, eight query heads) is cut into parts of equally many blocks, as many
// as there are warps to take them, which they do one after the other as they come free: CTAs whose SM still
// works on the prefix join in late.
// Weights go into the products in two bf16 parts (p - bf16(p) as well), or as one fp16.
//
// Measured: 64 sequences of 550 to 1,100 rows (217 MB) behind 16,384 (67 MB), 32 heads on 8 of 128: 70 us, 4.1 TB/s.  By
// themselves the rows behind take 46 us (4.8 TB/s), the prefix 39 us on half of the SMs, the join 12 us of a cold
// start: the first two run side by side, and the SMs of the prefix join in when it is done.  Small batches (8 sequences
// of 167 to 333 rows behind 2,048) 14.5 us: two dependent launches.
#pragma once
#include "attn16.cuh"

namespace g4 {

constexpr int kAttBlock = 16;      // rows of a block
constexpr int kAttMinPart = 4;     // blocks of a part at the least
constexpr int kAttMaxSeqs = 1024;

template <int D>
struct AttTail {
  static constexpr int kRows = kAttBlock * D * 2;                        // bytes of a block's keys, or values
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kWarps = D <= 128 ? 12 : D == 256 ? 6 : 3;        // 192 KB of rings
  static constexpr int kRing = kStages * 2 * kRows;
  static size_t smem(int n_seq) { return (size_t)kWarps * (kRing + 8 * kStages) + 16 + (size_t)(2 * n_seq + 1) * 4; }
};

struct AttTailArgs {
  const uint16_t *q, *kp, *vp;
  long q_row, q_head;
  uint16_t* out;
  long o_row, o_head;
  int o_vec;
  int n_seq, group, kvh, row_tiles;  // row_tiles: eights of query heads per KV head
  float scale;                       // times log2 e
  const int *table, *slots, *lens;
  int n_slots, n_pages, log_page, max_pages;
  int shared;                        // rows of the prefix that the slots share
  int keys;                          // and of the one that another kernel attends to: all of those, or none
  int most;                          // parts, but for one more of every item
  float* part_o;                     // [most + items][8][D]
  float2* part_ml;
  int4* plan;                        // of each sequence: its first part, parts of an item, error bits, rows
  unsigned* ticket;                  // [2]: the next part, CTAs that are done
  // the prefix's parts
  const float* pre_o;
  const float2* pre_ml;
  int splits, tb, blocks;            // tokens of a block of 128 rows, blocks of a part
  int* err;
};

// Rows behind the prefix that sequence i reads: 0 where its slot or length is not a valid one.
__device__ __forceinline__ int att_tail_len(const AttTailArgs& a, int i) {
  const int slot = __ldcg(a.slots + i);
  if (slot < 0 || slot >= a.n_slots) return 0;
  const int len = __ldcg(a.lens + slot);
  return len >= a.shared && len <= a.max_pages << a.log_page ? len - a.keys : 0;
}
// What is wrong with sequence i (error bits), and its rows; a warp's threads call it together.
__device__ __forceinline__ int att_check(const AttTailArgs& a, int i, int* rows) {
  const int lane = threadIdx.x & 31, slot = __ldcg(a.slots + i);
  *rows = 0;
  if (slot < 0 || slot >= a.n_slots) return G4_DEV_BAD_SLOT;
  const int len = __ldcg(a.lens + slot);
  if (len == 0) return 0;
  if (len < a.shared || len > a.max_pages << a.log_page) return G4_DEV_BAD_POSITION;
  const int shared = a.shared >> a.log_page, pages = (len + (1 << a.log_page) - 1) >> a.log_page;
  const int* table = a.table + (long)slot * a.max_pages;
  const int* same = a.table + (long)att_shared_slot(a.slots, a.lens, a.n_seq, a.n_slots, a.shared) * a.max_pages;  // (this slot at the latest)
  int wrong = 0;
#pragma unroll 4
  for (int p = lane; p < pages; p += 32) {
    const int id = __ldcg(table + p);
    wrong |= id < 0 || id >= a.n_pages || (p < shared && id != __ldcg(same + p));
  }
  *rows = len;
  return __any_sync(0xFFFFFFFFu, wrong) ? G4_DEV_BAD_POSITION : 0;
}

template <bool BF>
__device__ __forceinline__ void att_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t att_transpose(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, bool BF>
__global__ void __launch_bounds__(32 * AttTail<D>::kWarps, 1) att_tail_kernel(const AttTailArgs a) {
  using C = AttTail<D>;
  extern __shared__ __align__(16) uint8_t att_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = att_raw + warp * C::kRing;
  uint64_t* full = reinterpret_cast<uint64_t*>(att_raw + C::kWarps * C::kRing) + warp * C::kStages;
  int* shared = reinterpret_cast<int*>(att_raw + C::kWarps * (C::kRing + 8 * C::kStages));
  int* first = shared + 4;               // [n_seq + 1] parts ahead of each sequence
  int* lens = first + a.n_seq + 1;       // [n_seq]
  const int per_seq = a.kvh * a.row_tiles;
  if (lane < C::kStages) mbar_init(full + lane, 1);
  asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");

  // The arguments are older than the prefix's launch, which waited for what made them: they may be
  // read, and the rows attended to, while it runs.
  if (a.splits == 0) pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < a.n_seq; i += 32 * C::kWarps) lens[i] = att_tail_len(a, i);
  __syncthreads();
  if (warp == 0) {
    int blocks = 0;
    for (int i = lane; i < a.n_seq; i += 32) blocks += (lens[i] + kAttBlock - 1) / kAttBlock;
    const int total = (int)__reduce_add_sync(0xFFFFFFFFu, blocks) * per_seq;
    const int size = max(kAttMinPart, (total + a.most - 1) / a.most);  // blocks of a part
    int before = 0;
    for (int i0 = 0; i0 < a.n_seq; i0 += 32) {
      const int i = i0 + lane;
      int upto = i < a.n_seq ? ((lens[i] + kAttBlock - 1) / kAttBlock + size - 1) / size * per_seq : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += y;
      }
      if (i < a.n_seq) first[i + 1] = before + upto;
      before += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    if (lane == 0) {
      first[0] = 0;
      shared[0] = size;
    }
  }
  __syncthreads();
  const int total = first[a.n_seq], size = shared[0];
  bool alive = true;
  uint32_t used = 0;  // copies that were asked for: stage used % kStages
  for (int part = warp * gridDim.x + blockIdx.x; part < total && alive;) {  // (neighbours on different SMs)
    int lo = 0, hi = a.n_seq;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= part) lo = mid;
      else hi = mid;
    }
    const int seq = lo, len = lens[seq], blocks = (len + kAttBlock - 1) / kAttBlock, each = (blocks + size - 1) / size;
    const int x = (part - first[seq]) / each, from = (part - first[seq]) % each * size;
    const int head = x / a.row_tiles, row0 = x % a.row_tiles * 8, upto = min(blocks, from + size);
    const int* table = a.table + (long)__ldcg(a.slots + seq) * a.max_pages;

    // copy block b (a lane holds the page of block 32 k + lane of the part)
    int page = 0, pages_at = from;
    auto pages = [&](int at) {
      const int b = at + lane;
      page = b < upto ? __ldcg(table + ((a.keys + b * kAttBlock) >> a.log_page)) : 0;
      if (page < 0 || page >= a.n_pages) page = 0;  // (the join gives such a sequence zeros)
      pages_at = at;
    };
    auto copy = [&](int b) {
      if (b - pages_at >= 32) pages(b);
      const int pg = __shfl_sync(0xFFFFFFFFu, page, b - pages_at);
      if (lane == 0) {
        const int st = used % C::kStages, in = (a.keys + b * kAttBlock) & ((1 << a.log_page) - 1);
        const long at = ((((long)pg * a.kvh + head) << a.log_page) + in) * D;
        uint8_t* to = ring + st * 2 * C::kRows;
        mbar_expect_tx(full + st, 2 * C::kRows);
        bulk_g2s(to, a.kp + at, C::kRows, full + st);
        bulk_g2s(to + C::kRows, a.vp + at, C::kRows, full + st);
      }
      ++used;
    };
    pages(from);
    uint32_t next = used;  // the copy that is looked at next
#pragma unroll
    for (int i = 0; i < C::kStages; ++i)
      if (from + i < upto) copy(from + i);

    uint4 q[D / 32];  // row g, numbers 32 i + 8 t ..
    {
      const bool on = row0 + g < a.group;
      const uint16_t* p = a.q + (long)seq * a.q_row + (long)(head * a.group + (on ? row0 + g : 0)) * a.q_head + 8 * t;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) q[i] = on ? __ldcg(reinterpret_cast<const uint4*>(p + 32 * i)) : make_uint4(0u, 0u, 0u, 0u);
    }
    float o[D / 16][4];  // [16 numbers][number 0: rows 2t, 2t + 1; number 1]
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    for (int b = from; b < upto; ++b, ++next) {
      const int st = next % C::kStages;
      bool there = false;
      for (uint32_t i = 0; i < kSpinLimit && !there; ++i) there = mbar_try(full + st, (next / C::kStages) & 1);
      alive = __all_sync(0xFFFFFFFFu, there);
      if (!alive) {
        set_err(a.err, G4_DEV_TIMEOUT);
        break;
      }
      const uint8_t* kr = ring + st * 2 * C::kRows + g * (D * 2) + t * 16;
      const uint8_t* vr = ring + st * 2 * C::kRows + C::kRows + 2 * t * (D * 2) + g * 16;
      float c[4] = {0.f, 0.f, 0.f, 0.f}, d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 k0 = *reinterpret_cast<const uint4*>(kr + 64 * i), k1 = *reinterpret_cast<const uint4*>(kr + 16 * D + 64 * i);
        att_mma<BF>(c, k0.x, k1.x, k0.y, k1.y, q[i].x, q[i].y);
        att_mma<BF>(d, k0.z, k1.z, k0.w, k1.w, q[i].z, q[i].w);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = (c[i] + d[i]) * a.scale;
      const int live = len - b * kAttBlock;  // rows of the block that the sequence holds
      if (live < kAttBlock) {
        if (g >= live) c[0] = c[1] = -INFINITY;
        if (g + 8 >= live) c[2] = c[3] = -INFINITY;
      }
      // a row's reference is raised when a score exceeds it by 2^8 (attn16.cuh)
      const bool raise = fmaxf(c[0], c[2]) > m0 + 8.f || fmaxf(c[1], c[3]) > m1 + 8.f || m0 == -INFINITY || m1 == -INFINITY;
      if (__any_sync(0xFFFFFFFFu, raise)) {
        float x0 = fmaxf(c[0], c[2]), x1 = fmaxf(c[1], c[3]);
#pragma unroll
        for (int e = 4; e < 32; e <<= 1) {
          x0 = fmaxf(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, e));
          x1 = fmaxf(x1, __shfl_xor_sync(0xFFFFFFFFu, x1, e));
        }
        x0 = x0 > m0 + 8.f || m0 == -INFINITY ? fmaxf(m0, x0) : m0;
        x1 = x1 > m1 + 8.f || m1 == -INFINITY ? fmaxf(m1, x1) : m1;
        const float f0 = x0 == m0 ? 1.f : att_exp2(m0 - x0), f1 = x1 == m1 ? 1.f : att_exp2(m1 - x1);
        m0 = x0;
        m1 = x1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[i][0] *= f0;
          o[i][1] *= f1;
          o[i][2] *= f0;
          o[i][3] *= f1;
        }
      }
      const float z0 = m0 == -INFINITY ? 0.f : m0 - att_up<BF>(), z1 = m1 == -INFINITY ? 0.f : m1 - att_up<BF>();
      const float p0 = att_exp2(c[0] - z0), p1 = att_exp2(c[1] - z1), p2 = att_exp2(c[2] - z0), p3 = att_exp2(c[3] - z1);
      l0 += p0 + p2;
      l1 += p1 + p3;
      const uint32_t h0 = att_pack<BF>(p0, p1), h1 = att_pack<BF>(p2, p3);
      const uint32_t w0 = att_transpose(h0), w1 = att_transpose(h1);
      uint32_t r0 = 0, r1 = 0;
      if (BF) {
        r0 = att_transpose(att_pack<BF>(p0 - bf16_lo(h0), p1 - bf16_hi(h0)));
        r1 = att_transpose(att_pack<BF>(p2 - bf16_lo(h1), p3 - bf16_hi(h1)));
      }
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        uint4 v[4];  // rows 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const uint4*>(vr + ((e & 1) + (e >> 1) * 8) * (D * 2) + 128 * i);
        if (live < kAttBlock) {  // what lies behind the last row may be anything
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (2 * t + (e & 1) + (e >> 1) * 8 >= live) v[e] = make_uint4(0u, 0u, 0u, 0u);
        }
        const uint32_t* y0 = reinterpret_cast<const uint32_t*>(&v[0]);
        const uint32_t* y1 = reinterpret_cast<const uint32_t*>(&v[1]);
        const uint32_t* y2 = reinterpret_cast<const uint32_t*>(&v[2]);
        const uint32_t* y3 = reinterpret_cast<const uint32_t*>(&v[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t a0 = __byte_perm(y0[e], y1[e], 0x5410), a1 = __byte_perm(y0[e], y1[e], 0x7632);
          const uint32_t a2 = __byte_perm(y2[e], y3[e], 0x5410), a3 = __byte_perm(y2[e], y3[e], 0x7632);
          att_mma<BF>(o[i * 4 + e], a0, a1, a2, a3, w0, w1);
          if (BF) att_mma<BF>(o[i * 4 + e], a0, a1, a2, a3, r0, r1);
        }
      }
      __syncwarp();
      if (b + C::kStages < upto) copy(b + C::kStages);
    }
    unsigned mine = 0;
    if (lane == 0) mine = atomicAdd(a.ticket, 1u);
#pragma unroll
    for (int e = 4; e < 32; e <<= 1) {
      l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, e);
      l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, e);
    }
    if (lane < 4) {
      a.part_ml[(long)part * 8 + 2 * t] = make_float2(m0 - att_up<BF>(), l0);
      a.part_ml[(long)part * 8 + 2 * t + 1] = make_float2(m1 - att_up<BF>(), l1);
    }
    float* po = a.part_o + (long)part * 8 * D + g * 8;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      float4* even = reinterpret_cast<float4*>(po + (2 * t) * D + 64 * i);
      float4* odd = reinterpret_cast<float4*>(po + (2 * t + 1) * D + 64 * i);
      even[0] = make_float4(o[4 * i][0], o[4 * i][2], o[4 * i + 1][0], o[4 * i + 1][2]);
      even[1] = make_float4(o[4 * i + 2][0], o[4 * i + 2][2], o[4 * i + 3][0], o[4 * i + 3][2]);
      odd[0] = make_float4(o[4 * i][1], o[4 * i][3], o[4 * i + 1][1], o[4 * i + 1][3]);
      odd[1] = make_float4(o[4 * i + 2][1], o[4 * i + 2][3], o[4 * i + 3][1], o[4 * i + 3][3]);
    }
    part = gridDim.x * C::kWarps + (int)__shfl_sync(0xFFFFFFFFu, mine, 0);
  }
  if (!alive)  // what was asked for arrives before the CTA ends
    for (uint32_t k = used < C::kStages ? 0 : used - C::kStages; k < used; ++k) mbar_wait_drain(full + k % C::kStages, (k / C::kStages) & 1);
  // the sequences' checks and places, for the join
  for (int i = warp * gridDim.x + blockIdx.x; i < a.n_seq; i += gridDim.x * C::kWarps) {
    int rows;
    const int bad = att_check(a, i, &rows);
    if (lane == 0) {
      if (bad) set_err(a.err, bad);
      a.plan[i] = make_int4(first[i], (first[i + 1] - first[i]) / per_seq, bad, rows);
    }
  }
  if (a.splits) pdl_wait();  // so that who waits for this launch has waited for the prefix's too
  __syncthreads();
  if (threadIdx.x == 0) {  // the last CTA puts the counters back
    __threadfence();
    if (atomicAdd(a.ticket + 1, 1u) == gridDim.x - 1) {
      a.ticket[0] = 0;
      a.ticket[1] = 0;
    }
  }
}

constexpr int kAttJoinWarps = 4;

// The output of a query row from its parts: a CTA per row, its warps taking every fourth part (the prefix's
// before the rest's), whose sums are added in a fixed order.  A sequence that has been found wrong (att_check)
// gets zeros, and so does an empty one.
template <int D, bool BF>
__global__ void __launch_bounds__(32 * kAttJoinWarps) att_join_kernel(const AttTailArgs a) {
  constexpr int E = D / 32, R = E < 4 ? E : 4;  // numbers of a lane, in runs of 4 (2 at D = 64)
  __shared__ float sums[kAttJoinWarps][D];
  __shared__ float2 tops[kAttJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = a.kvh * a.group, seq = blockIdx.x / heads, hq = blockIdx.x % heads, head = hq / a.group, gr = hq % a.group;
  const int block = seq / a.tb, rows = a.blocks * kAttM;
  const long pre = ((long)(block / a.blocks) * a.kvh + head) * a.splits * rows + block % a.blocks * kAttM + seq % a.tb * a.group + gr;
  pdl_wait();
  pdl_trigger();
  const int4 plan = __ldcg(a.plan + seq);
  float acc[E], M = -INFINITY, L = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  if (!plan.z && plan.w > 0) {
    const int parts = a.splits + plan.y;
    const long own = (long)plan.x + (long)(head * a.row_tiles + gr / 8) * plan.y;
    // 32 of the warp's parts at a time: a lane looks at the maximum and sum of one
    for (int p0 = warp; p0 < parts; p0 += 32 * kAttJoinWarps) {
      const int p = p0 + lane * kAttJoinWarps;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (p < parts) ml = __ldcg(p < a.splits ? a.pre_ml + pre + (long)p * rows : a.part_ml + (own + p - a.splits) * 8 + gr % 8);
      const float top = fmaxf(M, warp_max(ml.x)), Z = top == -INFINITY ? 0.f : top;
      const float back = att_exp2(M - Z), mine = att_exp2(ml.x - Z);
      L = L * back + warp_sum(ml.y * mine);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= back;
      M = top;
      const int count = min(32, (parts - p0 + kAttJoinWarps - 1) / kAttJoinWarps);
#pragma unroll 4
      for (int i = 0; i < count; ++i) {
        const float f = __shfl_sync(0xFFFFFFFFu, mine, i);
        const int r = p0 + i * kAttJoinWarps;
        const float* o = r < a.splits ? a.pre_o + (pre + (long)r * rows) * D : a.part_o + ((own + r - a.splits) * 8 + gr % 8) * D;
#pragma unroll
        for (int e = 0; e < E; e += R) {
          if constexpr (R == 4) {
            const float4 u = __ldcg(reinterpret_cast<const float4*>(o + e * 32) + lane);
            acc[e] = fmaf(u.x, f, acc[e]);
            acc[e + 1] = fmaf(u.y, f, acc[e + 1]);
            acc[e + 2] = fmaf(u.z, f, acc[e + 2]);
            acc[e + 3] = fmaf(u.w, f, acc[e + 3]);
          } else {
            const float2 u = __ldcg(reinterpret_cast<const float2*>(o) + lane);
            acc[e] = fmaf(u.x, f, acc[e]);
            acc[e + 1] = fmaf(u.y, f, acc[e + 1]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < E; e += R)
#pragma unroll
    for (int k = 0; k < R; ++k) sums[warp][e * 32 + lane * R + k] = acc[e + k];
  if (lane == 0) tops[warp] = make_float2(M, L);
  __syncthreads();
  float top = tops[0].x;
#pragma unroll
  for (int w = 1; w < kAttJoinWarps; ++w) top = fmaxf(top, tops[w].x);
  if (top == -INFINITY) top = 0.f;
  float f[kAttJoinWarps], total = 0.f;
#pragma unroll
  for (int w = 0; w < kAttJoinWarps; ++w) {
    f[w] = att_exp2(tops[w].x - top);
    total = fmaf(tops[w].y, f[w], total);
  }
  const float inv = total != 0.f ? 1.f / total : 0.f;
  uint16_t* out = a.out + (long)seq * a.o_row + (long)hq * a.o_head;
  for (int c = 2 * threadIdx.x; c < D; c += 64 * kAttJoinWarps) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kAttJoinWarps; ++w) {
      x = fmaf(sums[w][c], f[w], x);
      y = fmaf(sums[w][c + 1], f[w], y);
    }
    const uint32_t u = att_pack<BF>(x * inv, y * inv);
    if (a.o_vec) {
      *reinterpret_cast<uint32_t*>(out + c) = u;
    } else {
      out[c] = (uint16_t)u;
      out[c + 1] = (uint16_t)(u >> 16);
    }
  }
}

}  // namespace g4
