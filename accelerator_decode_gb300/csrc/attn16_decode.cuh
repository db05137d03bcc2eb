// Attention of one token per sequence over a batch's rows behind their shared prefix, and the join of
// those parts with the prefix's (attn16.cuh).
//
// HBM bounds it: every row is read once, by a warp that keeps it in registers.  A block is 16 rows of
// one KV head, which lie in one page.  With the rows as the matrix instructions' 16-row operand and
// up to eight query heads as their columns,
//   S^T (16 keys x 8) = K Q^T     O^T (16 numbers x 8) += V^T P^T,
// a lane's 16-byte loads are its operands as they come: a permutation of the head dim that keys and
// queries share, and pairs of values' rows interleaved by a byte permutation.  O^T takes D / 4
// registers a lane.  All (sequence, KV head, block) triples are cut into equal spans, one per warp;
// an item (sequence, KV head, eight query heads) that lies in several spans leaves a part in each, so
// that few long rows use as many warps as many short ones.
// Weights go into the products in two bf16 parts (p - bf16(p) as well), or as one fp16.
#pragma once
#include "attn16.cuh"

namespace g4 {

constexpr int kAttBlock = 16;     // rows of a block
constexpr int kAttWarps = 4;      // warps of a CTA
constexpr int kAttMaxSeqs = 1024;

template <int D>
struct AttTail {
  static constexpr int kCtas = D <= 128 ? 4 : 2;                         // CTAs of an SM
  static constexpr int kQRow = D * 2 + 64;                               // bytes of a query row in shared memory
  static constexpr size_t kSmemQ = (size_t)kAttWarps * 8 * kQRow;
  static size_t smem(int n_seq) { return kSmemQ + (size_t)(2 * n_seq + 1) * 4; }
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
  int keys;                          // rows of the prefix
  float* part_o;                     // [2 * workers + items][8][D]
  float2* part_ml;
  int* plan;                         // [n_seq + 1] blocks ahead of each sequence, then the span
  int workers;
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
  return len >= a.keys && len <= a.max_pages << a.log_page ? len - a.keys : 0;
}
__device__ __forceinline__ int att_part(int worker, int t0, int span) { return 2 * worker + (t0 > worker * span); }

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
__device__ __forceinline__ uint4 att_stream(const uint16_t* p) {
  uint4 u;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
  return u;
}

template <int D, bool BF>
__global__ void __launch_bounds__(32 * kAttWarps, AttTail<D>::kCtas) att_tail_kernel(const AttTailArgs a) {
  using C = AttTail<D>;
  constexpr int KB = D / 32 < 8 ? D / 32 : 8, VB = D / 64 < 4 ? D / 64 : 4;  // pieces that a lane loads ahead
  extern __shared__ __align__(16) uint8_t att_raw[];
  int* first = reinterpret_cast<int*>(att_raw + C::kSmemQ);  // [n_seq + 1] blocks ahead, all heads counted
  int* lens = first + a.n_seq + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* sq = att_raw + warp * 8 * C::kQRow;
  const int per_block = a.kvh * a.row_tiles;

  // The arguments are older than the prefix's launch, which waited for what made them: they may be
  // read, and the rows attended to, while it runs.
  if (a.splits == 0) pdl_wait();
  pdl_trigger();
  if (warp == 0) {
    int before = 0;
    for (int i0 = 0; i0 < a.n_seq; i0 += 32) {
      const int i = i0 + lane, len = i < a.n_seq ? att_tail_len(a, i) : 0;
      int upto = (len + kAttBlock - 1) / kAttBlock * per_block;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += y;
      }
      if (i < a.n_seq) {
        first[i + 1] = before + upto;
        lens[i] = len;
      }
      before += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    if (lane == 0) first[0] = 0;
  }
  __syncthreads();
  const int total = first[a.n_seq], span = max(1, (total + a.workers - 1) / a.workers);
  const int me = blockIdx.x * kAttWarps + warp;
  const int b0 = (int)min((long)total, (long)me * span), b1 = min(total, b0 + span);
  for (int at = b0; at < b1;) {
    int lo = 0, hi = a.n_seq;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= at) lo = mid;
      else hi = mid;
    }
    const int seq = lo, len = lens[seq], blocks = (len + kAttBlock - 1) / kAttBlock;
    const int x = (at - first[seq]) / blocks, from = (at - first[seq]) % blocks, t0 = at - from;
    const int head = x / a.row_tiles, row0 = x % a.row_tiles * 8;
    const int upto = min(blocks, from + b1 - at);
    const int* table = a.table + (long)__ldcg(a.slots + seq) * a.max_pages;

    __syncwarp();
    for (int e = lane; e < 8 * (D / 8); e += 32) {  // the item's queries
      const int r = e / (D / 8), c = e % (D / 8);
      uint4 u = make_uint4(0u, 0u, 0u, 0u);
      if (row0 + r < a.group) {
        const uint16_t* p = a.q + (long)seq * a.q_row + (long)(head * a.group + row0 + r) * a.q_head + 8 * c;
        u = __ldcg(reinterpret_cast<const uint4*>(p));
      }
      *reinterpret_cast<uint4*>(sq + r * C::kQRow + c * 16) = u;
    }
    __syncwarp();

    float o[D / 16][4];  // [16 numbers][number 0: rows 2t, 2t + 1; number 1]
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    int page = __ldcg(table + ((a.keys + from * kAttBlock) >> a.log_page));
    for (int b = from; b < upto; ++b) {
      const int key = a.keys + b * kAttBlock, in = key & ((1 << a.log_page) - 1);
      if (page < 0 || page >= a.n_pages) page = 0;  // (the join gives such a sequence zeros)
      const long base = ((((long)page * a.kvh + head) << a.log_page) + in) * D;
      if (b + 1 < upto) page = __ldcg(table + ((key + kAttBlock) >> a.log_page));
      const uint16_t* kp = a.kp + base + g * D + t * 8;
      const uint16_t* vp = a.vp + base + 2 * t * D + g * 8;
      uint4 k[KB][2], v[VB][4];
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        k[i][0] = att_stream(kp + 32 * i);
        k[i][1] = att_stream(kp + 8 * D + 32 * i);
      }
#pragma unroll
      for (int i = 0; i < VB; ++i) {
        v[i][0] = att_stream(vp + 64 * i);
        v[i][1] = att_stream(vp + D + 64 * i);
        v[i][2] = att_stream(vp + 8 * D + 64 * i);
        v[i][3] = att_stream(vp + 9 * D + 64 * i);
      }
      float c[4] = {0.f, 0.f, 0.f, 0.f}, d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i0 = 0; i0 < D / 32; i0 += KB) {
#pragma unroll
        for (int i = 0; i < KB; ++i) {
          const uint4 u = *reinterpret_cast<const uint4*>(sq + g * C::kQRow + (i0 + i) * 64 + t * 16);
          att_mma<BF>(c, k[i][0].x, k[i][1].x, k[i][0].y, k[i][1].y, u.x, u.y);
          att_mma<BF>(d, k[i][0].z, k[i][1].z, k[i][0].w, k[i][1].w, u.z, u.w);
        }
        if (i0 + KB < D / 32) {
#pragma unroll
          for (int i = 0; i < KB; ++i) {
            k[i][0] = att_stream(kp + 32 * (i0 + KB + i));
            k[i][1] = att_stream(kp + 8 * D + 32 * (i0 + KB + i));
          }
        }
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
      const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
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
      for (int i0 = 0; i0 < D / 64; i0 += VB) {
        if (live < kAttBlock) {  // what lies behind the last row may be anything
#pragma unroll
          for (int i = 0; i < VB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (2 * t + (e & 1) + (e >> 1) * 8 >= live) v[i][e] = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < VB; ++i) {
          const uint32_t* y0 = reinterpret_cast<const uint32_t*>(&v[i][0]);
          const uint32_t* y1 = reinterpret_cast<const uint32_t*>(&v[i][1]);
          const uint32_t* y2 = reinterpret_cast<const uint32_t*>(&v[i][2]);
          const uint32_t* y3 = reinterpret_cast<const uint32_t*>(&v[i][3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t a0 = __byte_perm(y0[e], y1[e], 0x5410), a1 = __byte_perm(y0[e], y1[e], 0x7632);
            const uint32_t a2 = __byte_perm(y2[e], y3[e], 0x5410), a3 = __byte_perm(y2[e], y3[e], 0x7632);
            att_mma<BF>(o[(i0 + i) * 4 + e], a0, a1, a2, a3, w0, w1);
            if (BF) att_mma<BF>(o[(i0 + i) * 4 + e], a0, a1, a2, a3, r0, r1);
          }
        }
        if (i0 + VB < D / 64) {
#pragma unroll
          for (int i = 0; i < VB; ++i) {
            const uint16_t* p = vp + 64 * (i0 + VB + i);
            v[i][0] = att_stream(p);
            v[i][1] = att_stream(p + D);
            v[i][2] = att_stream(p + 8 * D);
            v[i][3] = att_stream(p + 9 * D);
          }
        }
      }
    }
#pragma unroll
    for (int e = 4; e < 32; e <<= 1) {
      l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, e);
      l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, e);
    }
    const bool whole = from == 0 && upto == blocks;
    const long part = whole ? 2L * a.workers + (long)seq * per_block + x : att_part(me, t0, span);
    if (lane < 4) {
      a.part_ml[part * 8 + 2 * t] = make_float2(m0, l0);
      a.part_ml[part * 8 + 2 * t + 1] = make_float2(m1, l1);
    }
    float* po = a.part_o + part * 8 * D + g * 8;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      float4* even = reinterpret_cast<float4*>(po + (2 * t) * D + 64 * i);
      float4* odd = reinterpret_cast<float4*>(po + (2 * t + 1) * D + 64 * i);
      even[0] = make_float4(o[4 * i][0], o[4 * i][2], o[4 * i + 1][0], o[4 * i + 1][2]);
      even[1] = make_float4(o[4 * i + 2][0], o[4 * i + 2][2], o[4 * i + 3][0], o[4 * i + 3][2]);
      odd[0] = make_float4(o[4 * i][1], o[4 * i][3], o[4 * i + 1][1], o[4 * i + 1][3]);
      odd[1] = make_float4(o[4 * i + 2][1], o[4 * i + 2][3], o[4 * i + 3][1], o[4 * i + 3][3]);
    }
    at = t0 + upto;
  }
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i <= a.n_seq; i += 32 * kAttWarps) a.plan[i] = first[i];
    if (threadIdx.x == 0) a.plan[a.n_seq + 1] = span;
  }
  if (a.splits) pdl_wait();  // so that who waits for this launch has waited for the prefix's too
}

// The output of a query row from its parts: a warp per row, the prefix's parts before the rest's.  A
// sequence whose slot, length or pages are not valid ones, or whose first pages are not the shared ones,
// gets zeros, with the error word set (an empty one without).
template <int D, bool BF>
__global__ void __launch_bounds__(256) att_join_kernel(const AttTailArgs a) {
  const int lane = threadIdx.x & 31, r = blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  const int heads = a.kvh * a.group;
  if (r >= a.n_seq * heads) return;
  const int seq = r / heads, hq = r % heads, head = hq / a.group, gr = hq % a.group;
  const int slot = __ldcg(a.slots + seq);
  int bad = slot < 0 || slot >= a.n_slots ? G4_DEV_BAD_SLOT : 0, len = 0;
  if (!bad) {
    len = __ldcg(a.lens + slot);
    if (len < 0 || len > a.max_pages << a.log_page || (len > 0 && len < a.keys)) bad = G4_DEV_BAD_POSITION;
  }
  if (!bad && len > 0) {
    const int* table = a.table + (long)slot * a.max_pages;
    const int shared = a.keys >> a.log_page, pages = (len + (1 << a.log_page) - 1) >> a.log_page;
    const int* same = a.table + (long)att_shared_slot(a.slots, a.lens, a.n_seq, a.n_slots, a.keys) * a.max_pages;  // (this slot at the latest)
    int wrong = 0;
#pragma unroll 4
    for (int p = lane; p < pages; p += 32) {
      const int id = __ldcg(table + p);
      wrong |= id < 0 || id >= a.n_pages || (p < shared && id != __ldcg(same + p));
    }
    if (__any_sync(0xFFFFFFFFu, wrong)) bad = G4_DEV_BAD_POSITION;
  }
  if (bad && lane == 0 && gr == 0 && head == 0) set_err(a.err, bad);
  uint16_t* out = a.out + (long)seq * a.o_row + (long)hq * a.o_head;
  constexpr int E = D / 32;  // numbers of a lane, in runs of 4 (2 at D = 64)
  constexpr int R = E < 4 ? E : 4;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float inv = 0.f;
  if (!bad && len > 0) {
    const int block = seq / a.tb, rows = a.blocks * kAttM;
    const long pre = ((long)(block / a.blocks) * a.kvh + head) * a.splits * rows + block % a.blocks * kAttM + seq % a.tb * a.group + gr;
    const int x = head * a.row_tiles + gr / 8, b0 = __ldcg(a.plan + seq), span = __ldcg(a.plan + a.n_seq + 1);
    const int blocks = (len - a.keys + kAttBlock - 1) / kAttBlock, t0 = b0 + x * blocks;
    const int c0 = t0 / span, c1 = blocks ? (t0 + blocks - 1) / span : c0 - 1;
    const int own = c1 - c0 + 1, parts = a.splits + own;
    auto row_of = [&](int p, const float2** ml, const float** o) {
      if (p < a.splits) {
        const long at = pre + (long)p * rows;
        *ml = a.pre_ml + at;
        *o = a.pre_o + at * D;
      } else {
        const int c = c0 + p - a.splits;
        const long at = (own == 1 ? 2L * a.workers + (long)seq * a.kvh * a.row_tiles + x : (long)att_part(c, t0, span)) * 8 + gr % 8;
        *ml = a.part_ml + at;
        *o = a.part_o + at * D;
      }
    };
    const float2* ml;
    const float* o;
    float M = -INFINITY;
    for (int p = lane; p < parts; p += 32) {
      row_of(p, &ml, &o);
      M = fmaxf(M, __ldcg(&ml->x));
    }
    M = warp_max(M);
    if (M == -INFINITY) M = 0.f;
    float L = 0.f;
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      row_of(p, &ml, &o);
      const float2 w = __ldcg(ml);
      const float f = att_exp2(w.x - M);
      L = fmaf(w.y, f, L);
#pragma unroll
      for (int e = 0; e < E; e += R) {
        if (R == 4) {
          const float4 u = __ldcg(reinterpret_cast<const float4*>(o + e * 32) + lane);
          acc[e] = fmaf(u.x, f, acc[e]);
          acc[e + 1] = fmaf(u.y, f, acc[e + 1]);
          acc[e + 2 < E ? e + 2 : 0] = fmaf(u.z, f, acc[e + 2 < E ? e + 2 : 0]);
          acc[e + 3 < E ? e + 3 : 0] = fmaf(u.w, f, acc[e + 3 < E ? e + 3 : 0]);
        } else {
          const float2 u = __ldcg(reinterpret_cast<const float2*>(o) + lane);
          acc[e] = fmaf(u.x, f, acc[e]);
          acc[e + 1] = fmaf(u.y, f, acc[e + 1]);
        }
      }
    }
    inv = L != 0.f ? 1.f / L : 0.f;
  }
#pragma unroll
  for (int e = 0; e < E; e += R) {
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < R / 2; ++k) w[k] = att_pack<BF>(acc[e + 2 * k] * inv, acc[e + 2 * k + 1] * inv);
    uint16_t* to = out + e * 32 + lane * R;
    if (a.o_vec) {
      if (R == 4) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(to) = w[0];
    } else {
#pragma unroll
      for (int k = 0; k < R / 2; ++k) {
        to[2 * k] = (uint16_t)w[k];
        to[2 * k + 1] = (uint16_t)(w[k] >> 16);
      }
    }
  }
}

}  // namespace g4
