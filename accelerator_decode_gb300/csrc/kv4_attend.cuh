// Softmax attention over the 4-bit cache (kv4.cuh), and the account of attention weights.
//
//   s_j = scale q . K_j      o = sum_j softmax(s)_j V_j      account_j += sum over (t, head) softmax(s)_j
// for the rows j that query token t sees: j <= len - m + t, and j > len - m + t - window.
//
// Work: an item is eight query rows (query token x head, all of one KV head) against the rows
// of their sequence.  All items' key tiles, laid end to end, are cut into equal spans, one per
// CTA, so a ragged batch or a single long sequence fills the GPU alike; a span's first and last
// item may be shared with the neighbouring CTAs, which leave partial sums.  Those are joined by
// the CTA that finishes an item last (few parts an item), or by kv4_finish_kernel.
//
// Per CTA one producer warp (D = 512: the first consumer warp) streams key tiles into a
// shared-memory ring with bulk copies; each consumer warp takes whole blocks of 16 keys through scores, running softmax and output with
// no synchronisation with the other warps until the item ends.  Both products run on the tensor
// cores with the cache as the M operand (m16n8k16: 16 keys, or 16 numbers of the value, by 8
// query rows), so eight query rows of a KV head fill the N operand (four leave half of it empty), and
// 4-bit codes go from a 16-byte load to the operand registers through 1.25 ALU operations and one
// bf16 operation per pair.
//
// Bound: the dependent chain of a block (load, decode, scores, softmax, values), with 8 to 12
// consumer warps on an SM to hide it.  64 sequences of up to 8,192 rows, eight KV heads of 128, four
// query heads each (456 MB, 68 us at the measured copy rate): 109 us, 4.2 TB/s; loading alone takes 88
// us and the arithmetic on resident tiles 107.  At 16 sequences the issue slots are 48% busy, the
// tensor cores 26%, DRAM 37%.  512-wide rows, eight sequences of up to 8,639: bf16 33 us (17% of the
// issue slots, 9% of the tensor cores, DRAM 11%), fp32 40; of the 11 cycles between a warp's
// instructions 3.5 wait for instruction fetches and 2.5 at barriers, three tiles a warp.  64 windows of
// 512 rows of 256, fp32: 13 us and 7 for the join, two tiles a CTA.  One sequence of 200 rows: 11 us; of a
// cold launch half are instruction fetches and a fifth barriers.
//
// The output's sums fill the registers.  Compiled, the 128-wide kernels spill 160 (fp32) and 24 (fp16)
// bytes of their 128 registers a thread, the 64-wide fp32 one 20, the others none.
#pragma once
#include "kv4.cuh"
#include "mbar.cuh"

namespace g4 {

struct Kv4AttendArgs {
  Kv4Cache c;
  const int *slots, *lens, *q_lens;  // q_lens may be NULL
  int n_seq, q_len, heads, group;    // group: query heads per KV head
  int row_tiles;                     // items of a (sequence, KV head): ceil(q_len * group / 8)
  float scale;                       // times log2(e)
  int plain;                         // codes are decoded as in a cache with wide scales: scale * 2^64 is infinite
  int window, accumulate, zero_rest;
  int join_inside;                   // the CTA that finishes a shared item last joins its parts
  int stages;
  Kv4Dense q, out;
  float* lse;                        // [n_seq][kvh][lse_rows]: log2 of the softmax's sum
  int lse_rows;
  float4* part_o;                    // [2 * CTAs][D / 32][2][32]: a span's partial first and last item
  float2* part_ml;                   // [2 * CTAs][8]: running maximum (log2 units) and sum
  unsigned* tickets;                 // [items]: parts done, zero between calls
};

// Sequence i's slot, rows and query tokens; false (uniform over the block) when it is skipped.
__device__ __forceinline__ bool kv4_seq(const Kv4AttendArgs& a, int i, int* slot, int* len, int* m) {
  *slot = __ldcg(a.slots + i);
  *len = __ldcg(a.lens + i);
  *m = a.q_lens ? __ldcg(a.q_lens + i) : a.q_len;
  return *slot >= 0 && *slot < a.c.n_slots && *len >= 0 && *len <= a.c.capacity && *m >= 0 && *m <= a.q_len;
}
// Error bits of a skipped sequence.
__device__ __forceinline__ int kv4_seq_error(const Kv4AttendArgs& a, int slot) {
  return slot < 0 || slot >= a.c.n_slots ? G4_DEV_BAD_SLOT : G4_DEV_BAD_POSITION;
}

__device__ __forceinline__ void named_bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}
// A whole warp's bounded wait, with one answer for all its lanes: each lane counts and looks at the
// abort flag for itself, and lanes that went on with different answers would meet the votes and
// shuffles behind the wait without each other.
__device__ __forceinline__ bool kv4_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag));
  if (!ok) *abort_flag = 1;
  return ok;
}
// 2^x, relative error 2^-22; 0 for -inf.  Its argument is a score minus a reference (a maximum, or the
// log2 of a sum) that was itself taken of rounded scores, so the score is rounded before the
// subtraction (__fmul_rn).  A fused multiply-subtract gives back what the rounding took, up to 2^-24
// of the score: a weight of 1 became 1.03 at scores of 2^19, and infinite from 2^31 on.
__device__ __forceinline__ float kv4_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// D (16 x 8, fp32) += A (16 x 16, bf16) B (16 x 8, bf16)
__device__ __forceinline__ void kv4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t kv4_transpose(uint32_t x) {  // 8 x 8 matrix of 16-bit numbers
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
// x = the bf16 numbers of `parts` registers added up: the first takes x's top 8 bits, each next
// one 8 of the rest.  bf16 queries need one part, fp16 two (11 bits), fp32 three (24 bits); a
// softmax weight two (2^-17 of it, against an output rounded at 2^-9 or 2^-12) or, for fp32
// outputs, three.
template <int PARTS>
__device__ __forceinline__ void kv4_split(float x, float y, uint32_t (&p)[PARTS]) {
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    p[i] = as_u32(h);
    if (i + 1 < PARTS) {
      x -= bf16_lo(p[i]);
      y -= bf16_hi(p[i]);
    }
  }
}

constexpr int kKv4MaxCtas = 3;

template <int D, int DT>
struct Kv4Att {
  static constexpr int kQP = DT == G4_DT_F32 ? 3 : DT == G4_DT_F16 ? 2 : 1;  // parts of a query
  static constexpr int kPP = DT == G4_DT_F32 ? 3 : 2;                       // parts of a weight
  static constexpr int kWarps = D == 512 ? 8 : 4;      // consumer warps
  static constexpr int kSets = kWarps / 4;             // sets of four warps take tiles in turn
  static constexpr int kBpw = D >= 256 ? 1 : 256 / D;  // blocks a warp takes of a tile
  static constexpr int kBlocks = 4 * kBpw;             // blocks of a tile
  static constexpr int kNB = kBpw;                     // blocks a warp takes through the softmax at a time
  static constexpr int kKeys = kBlocks * kKv4Block;    // keys of a tile: 256, 128, 64, 64
  static constexpr int kTile = kBlocks * 18 * D;       // bytes of a tile: 18 KB (D = 512: 36 KB)
  // D = 512: the first consumer warp fills the ring as well.  A ninth warp would put three on one
  // scheduler and so leave 168 registers a thread, and the 128 of the output would spill.
  static constexpr bool kOwnProducer = D != 512;
  static constexpr int kThreads = 32 * (kWarps + (kOwnProducer ? 1 : 0));
  static constexpr int kMinCtas = D == 512 ? 1 : D == 256 ? 2 : 3;  // CTAs of an SM
  static_assert(kMinCtas <= kKv4MaxCtas, "the partial sums' buffers hold two items of so many CTAs per SM");
  static constexpr int kQBytes = kQP * D * 16;         // [part][D / 32][lane] 16-byte pieces
  // Warps whose sums fit in shared memory at a time.  At D = 512 four regions leave the ring four
  // stages with bf16 queries, and with fp16 ones up to 114 sequences (three are not sound,
  // kv4_ring_stages: then two); fp32 queries have four stages beside two regions only, whose sums take
  // one more round at an item's end.  Four / two regions, microseconds: bf16, eight sequences of 8,639
  // rows 43.1 / 45.0; fp16, eight of those without the account 39.3 / 40.9, 64 of 640 rows 27.4 /
  // 28.7, 128 of them 55.5 / 49.2.
  static constexpr int kRegions = D == 256 || (D == 512 && DT != G4_DT_F32) ? 4 : 2;
  static constexpr int kOBytes = kRegions * D * 32;    // [region][D / 32][2][lane] float4
  static_assert(kOBytes >= kKv4MaxSlots * 4, "the plan's table of slots lies where the sums will");
  static constexpr int kFixed = kQBytes + kOBytes + kWarps * 64 + 256;  // + running (max, sum) of every warp, barriers
  static __host__ __device__ size_t smem(int stages, int n_seq) {
    return (size_t)stages * kTile + kFixed + (size_t)n_seq * 20 + 16;
  }
};

// The cut of all tiles into spans, worked out by every CTA for itself: first[i] = key tiles of all
// items of sequences before i (sequence i has kvh * row_tiles items of the same number of tiles),
// first[n_seq + 1] = tiles of the longest item; seqs[i] = (slot, len, m), len 0 when skipped.
template <int KEYS>
__device__ __forceinline__ int kv4_tiles(const Kv4AttendArgs& a, int len, int m, int* tile0) {
  const int lo = a.window > 0 ? max(0, len - m + 1 - a.window) : 0;  // first row that token 0 sees
  *tile0 = lo / KEYS;
  return m > 0 && len > 0 ? (len + KEYS - 1) / KEYS - *tile0 : 0;
}
// owner: shared scratch of one int per slot, for a call that accumulates: the first sequence that
// names it.  (Each sequence looking through the ones before it, in every CTA, took 38 ms with 1,024
// sequences.)
template <int KEYS>
__device__ __forceinline__ void kv4_plan(const Kv4AttendArgs& a, int* first, int4* seqs, int* owner, bool report) {
  if (a.accumulate) {
    for (int s = threadIdx.x; s < a.c.n_slots; s += blockDim.x) owner[s] = a.n_seq;
    __syncthreads();
    for (int i = threadIdx.x; i < a.n_seq; i += blockDim.x) {
      const int slot = __ldcg(a.slots + i);
      if (slot >= 0 && slot < a.c.n_slots) atomicMin(owner + slot, i);
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < a.n_seq; i += blockDim.x) {
    int slot, len, m, t0;
    bool ok = kv4_seq(a, i, &slot, &len, &m);
    if (!ok && report) set_err(a.c.err, kv4_seq_error(a, slot));
    if (a.accumulate && ok && owner[slot] != i) {  // a slot that an earlier sequence names is skipped
      if (report) set_err(a.c.err, G4_DEV_BAD_SLOT);
      len = 0;
    }
    if (!ok) {  // all its query rows get zeros
      len = 0;
      m = a.q_len;
    }
    seqs[i] = make_int4(slot, len, m, kv4_tiles<KEYS>(a, len, m, &t0));
  }
  __syncthreads();
  if (threadIdx.x < 32) {  // running sum, 32 sequences at a time
    const int lane = threadIdx.x;
    int base = 0;
    int longest = 0;
    if (lane == 0) first[0] = 0;
    for (int i = 0; i < a.n_seq; i += 32) {
      const int n = i + lane < a.n_seq ? seqs[i + lane].w : 0;
      longest = max(longest, n);
      int v = n * a.c.kvh * a.row_tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
      }
      if (i + lane < a.n_seq) first[i + lane + 1] = base + v;
      base += __shfl_sync(0xFFFFFFFFu, v, 31);
    }
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    if (lane == 0) first[a.n_seq + 1] = longest;
  }
  __syncthreads();
}
// Tiles per CTA.  An item that is joined inside is shared by kKv4Join + 1 CTAs at the most (4 and 16
// measure the same within 2%, where items are many or few).
constexpr int kKv4Join = 8;
__device__ __forceinline__ int kv4_span(const Kv4AttendArgs& a, const int* first, int ctas) {
  const int even = (int)(((unsigned)first[a.n_seq] + ctas - 1) / ctas);
  return max(1, a.join_inside ? max(even, (first[a.n_seq + 1] + kKv4Join - 1) / kKv4Join) : even);
}

// A run of tiles of one item: what a CTA does between two item borders.
struct Kv4Run {
  int seq, head, row_tile;
  int slot, len, m;
  int tile, tiles;     // first tile (absolute) and their number
  int of;              // tiles of the item
  int item_t0;   // the item's first tile in the order of all
  bool whole;          // the run is the whole item
};
// The run that starts at global tile g (g < end <= total).
template <int KEYS>
__device__ __forceinline__ Kv4Run kv4_run(const Kv4AttendArgs& a, const int* first, const int4* seqs, int g, int end) {
  int lo = 0, hi = a.n_seq - 1;  // the last sequence with first[i] <= g (empty ones in between share it)
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (first[mid] <= g) lo = mid; else hi = mid - 1;
  }
  Kv4Run r;
  r.seq = lo;
  const int4 q = seqs[lo];
  r.slot = q.x;
  r.len = q.y;
  r.m = q.z;
  r.of = q.w;
  int t0;
  kv4_tiles<KEYS>(a, r.len, r.m, &t0);
  const int x = g - first[lo];
  const int item = (unsigned)x / (unsigned)r.of, off = x - item * r.of;
  r.item_t0 = g - off;
  r.head = item / a.row_tiles;
  r.row_tile = item % a.row_tiles;
  r.tile = t0 + off;
  r.tiles = min(r.of - off, end - g);
  r.whole = r.tiles == r.of;
  return r;
}

// ------------------------------------------------------------------------- the pieces
// Queries of rows row0 .. row0 + 7 of (sequence, KV head) as bf16 parts in the order of the mma's
// B operand: piece (part, w) of lane l is row l / 4, numbers (l % 4) D/4 + 8w .. + 7.
template <int D, int DT>
__device__ __forceinline__ void kv4_stage_q(const Kv4AttendArgs& a, uint4* qs, int seq, int head, int row0, int n_rows,
                                            int tid, int threads) {
  constexpr int W = D / 32, QP = Kv4Att<D, DT>::kQP;
  for (int e = tid; e < W * 32; e += threads) {
    const int w = e >> 5, l = e & 31, row = row0 + (l >> 2);
    float v[8];
    if (row < n_rows) {
      const int tok = row / a.group, hq = head * a.group + row % a.group;
      kv4_load8(a.q, (long)seq * a.q.seq + (long)tok * a.q.row + (long)hq * a.q.head + (l & 3) * (D / 4) + 8 * w, v);
    } else {
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = 0.f;
    }
    uint32_t p[4][QP];
#pragma unroll
    for (int x = 0; x < 4; ++x) kv4_split<QP>(v[2 * x], v[2 * x + 1], p[x]);
#pragma unroll
    for (int part = 0; part < QP; ++part) qs[(part * W + w) * 32 + l] = make_uint4(p[0][part], p[1][part], p[2][part], p[3][part]);
  }
}

// The scales of one key's numbers that lane t holds, [t D/4, (t+1) D/4): one bf16 per 32 of them
// (D = 64: of half a group).  two(k): the k-th in both halves of a bf16x2.
template <int D>
struct Kv4KeyScales {
  static constexpr int N = D >= 128 ? D / 128 : 1;
  uint32_t raw[(N + 1) / 2];
  __device__ __forceinline__ uint32_t two(int k) const { return __byte_perm(raw[k >> 1], 0u, k & 1 ? 0x3232u : 0x1010u); }
};
template <int D>
__device__ __forceinline__ Kv4KeyScales<D> kv4_key_scales(const uint8_t* ks, int key, int t) {
  Kv4KeyScales<D> r;
  const uint8_t* p = ks + key * (D / 16) + (D >= 128 ? t * (D / 64) : (t >> 1) * 2);
  if constexpr (D == 512) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    r.raw[0] = u.x;
    r.raw[1] = u.y;
  } else if constexpr (D == 256) {
    r.raw[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    r.raw[0] = *reinterpret_cast<const uint16_t*>(p);
  }
  return r;
}

// Scores of NB blocks of 16 keys by eight query rows, summed over the head dim (before the
// softmax scale): c[b] in the mma's accumulator order.  codes(b, i): 16-byte piece i of block b;
// scales(b, half): scales of key g + 8 half.
template <int D, int QP, int NB, bool WIDE, class Codes, class Scales>
__device__ __forceinline__ void kv4_scores(const uint4* qs, int lane, Codes codes, Scales scales, float (&c)[NB][4]) {
  constexpr int W = D / 32, N = Kv4KeyScales<D>::N;
  float d[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[b][j] = d[b][j] = 0.f;
#pragma unroll
  for (int grp = 0; grp < N; ++grp) {  // a lane's numbers of one group: W / 2 / N pieces
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const Kv4Scale<WIDE> sg(scales(b, 0).two(grp)), sh(scales(b, 1).two(grp));
#pragma unroll
      for (int i = grp * (W / 2 / N); i < (grp + 1) * (W / 2 / N); ++i) {
        const uint4 u = codes(b, i);  // row g: words 2i, 2i + 1; row g + 8: same
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t ug = e ? u.y : u.x, uh = e ? u.w : u.z;
          const uint32_t a0 = sg.template pair<0>(ug), a1 = sh.template pair<0>(uh), a2 = sg.template pair<1>(ug), a3 = sh.template pair<1>(uh);
          const uint32_t b0 = sg.template pair<2>(ug), b1 = sh.template pair<2>(uh), b2 = sg.template pair<3>(ug), b3 = sh.template pair<3>(uh);
#pragma unroll
          for (int part = 0; part < QP; ++part) {
            const uint4 qv = qs[(part * W + 2 * i + e) * 32 + lane];
            kv4_mma(c[b], a0, a1, a2, a3, qv.x, qv.y);
            kv4_mma(d[b], b0, b1, b2, b3, qv.z, qv.w);
          }
        }
      }
    }
  }
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[b][j] += d[b][j];
}

// What the warps of a CTA share.
template <int D, int DT>
struct Kv4Shared {
  uint8_t* ring;
  uint4* qs;
  float4* os;
  float2* mls;        // [warp][8]
  uint64_t *full, *empty;
  uint32_t* held;     // [8]: blocks of a stage that hold rows
  volatile int* abort_flag;
  volatile int* last;  // this CTA joins the item
  int4* seqs;
  int* first;
  __device__ __forceinline__ Kv4Shared(uint8_t* smem, int stages, int n_seq) {
    using C = Kv4Att<D, DT>;
    ring = smem;
    qs = reinterpret_cast<uint4*>(ring + (size_t)stages * C::kTile);
    os = reinterpret_cast<float4*>(reinterpret_cast<uint8_t*>(qs) + C::kQBytes);
    mls = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(os) + C::kOBytes);
    full = reinterpret_cast<uint64_t*>(mls + C::kWarps * 8);
    empty = full + 8;
    held = reinterpret_cast<uint32_t*>(empty + 8);
    abort_flag = reinterpret_cast<volatile int*>(held + 8);
    last = abort_flag + 1;
    seqs = reinterpret_cast<int4*>(full + 32);
    first = reinterpret_cast<int*>(seqs + n_seq);
  }
};

// ------------------------------------------------------------------------ joining parts
// CTA c's part of the item that starts at tile t0: slot 0 when the item opens c's span, else 1.
__device__ __forceinline__ long kv4_part(int c, int t0, int span) { return (long)c * 2 + (t0 > c * span ? 1 : 0); }
__device__ __forceinline__ float kv4_lse(float2 ml) { return ml.y != 0.f ? ml.x + log2f(ml.y) : INFINITY; }
__device__ __forceinline__ void kv4_merge_ml(float2& u, float2 v) {
  const float m = fmaxf(u.x, v.x), z = m == -INFINITY ? 0.f : m;
  u.y = u.y * kv4_exp2(u.x - z) + v.y * kv4_exp2(v.x - z);
  u.x = m;
}
// Maximum and sum of the item's eight rows over its parts c0 .. c1 into ml[0..8), by `warps` warps
// that share barrier `bar` (ml: 8 + 8 * warps entries): a thread takes a row and every 4 warps'th part.
__device__ __forceinline__ void kv4_join_ml(const Kv4AttendArgs& a, int t0, int span, int c0, int c1, int tid,
                                            int warps, float2* ml, int bar) {
  float2 u = make_float2(-INFINITY, 0.f);
#pragma unroll 4
  for (int c = c0 + (tid >> 3); c <= c1; c += 4 * warps) kv4_merge_ml(u, __ldcg(&a.part_ml[kv4_part(c, t0, span) * 8 + (tid & 7)]));
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    const float2 v = make_float2(__shfl_xor_sync(0xFFFFFFFFu, u.x, o), __shfl_xor_sync(0xFFFFFFFFu, u.y, o));
    kv4_merge_ml(u, v);
  }
  if ((tid & 31) < 8) ml[8 + (tid >> 5) * 8 + (tid & 7)] = u;
  named_bar_sync(bar, 32 * warps);
  if (tid < 8) {
    u = ml[8 + tid];
    for (int w = 1; w < warps; ++w) kv4_merge_ml(u, ml[8 + w * 8 + tid]);
    ml[tid] = u;
  }
  named_bar_sync(bar, 32 * warps);
}
// The item's output rows from its parts, in span order; entries e0, e0 + step, ..  Eight parts'
// loads are in flight at a time (one after the other they cost a round trip each: 12,000 cycles
// for four parts of a 256-wide item).
template <int D>
__device__ __forceinline__ void kv4_join_rows(const Kv4AttendArgs& a, int seq, int head, int row0, int n_rows, int t0,
                                              int span, int c0, int c1, const float2* ml, int e0, int step) {
  constexpr int W = D / 32;
  for (int e = e0; e < W * 64; e += step) {
    const int l = e & 31, r8 = 2 * (l & 3) + ((e >> 5) & 1), w = e >> 6, row = row0 + r8;
    const float M = ml[r8].x, Z = M == -INFINITY ? 0.f : M, L = ml[r8].y, inv = L != 0.f ? 1.f / L : 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int cb = c0; cb <= c1; cb += 8) {
      float4 u[8];
      float f[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (cb + q <= c1) {
          const long p = kv4_part(cb + q, t0, span);
          f[q] = __ldcg(&a.part_ml[p * 8 + r8].x);
          u[q] = __ldcg(&a.part_o[p * W * 64 + e]);
        }
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (cb + q <= c1) {
          const float x = kv4_exp2(f[q] - Z);
          v.x += x * u[q].x;
          v.y += x * u[q].y;
          v.z += x * u[q].z;
          v.w += x * u[q].w;
        }
      }
    }
    if (row < n_rows) {
      const int tok = row / a.group, hq = head * a.group + row % a.group;
      kv4_store4(a.out, (long)seq * a.out.seq + (long)tok * a.out.row + (long)hq * a.out.head + (l >> 2) * (D / 8) + 4 * w,
                 make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
    }
  }
}
// The same by a CTA's consumer warps once their ring is idle: the parts come through it, all in
// flight together, and the rolled loops keep the code short.  (Code that runs once a launch costs
// its fetching: a join unrolled over the parts was slower than one round trip after the other.)
// Also writes the rows' lse.
template <int D, int DT>
__device__ __forceinline__ void kv4_join_ring(const Kv4AttendArgs& a, const Kv4Shared<D, DT>& sh, const Kv4Run& r, int span, int c0, int c1, float* lse) {
  using C = Kv4Att<D, DT>;
  constexpr int E = D * 2, T = 32 * C::kWarps, N = E / T;  // 16-byte entries of a part, and of a thread
  float2* ml = reinterpret_cast<float2*>(sh.os);           // [part][8]
  float4* buf = reinterpret_cast<float4*>(sh.ring);
  const int tid = threadIdx.x, n = c1 - c0 + 1, cap = a.stages * C::kTile / (E * 16);
  const int l = tid & 31, r8 = 2 * (l & 3) + ((tid >> 5) & 1);  // the same row in all of a thread's entries
  float4 v[N];
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, L = 0.f;
  for (int p0 = 0; p0 < n; p0 += cap) {
    const int np = min(cap, n - p0);
    if (p0) named_bar_sync(1, T);
    for (int c = 0; c < np; ++c) {
      const float4* from = a.part_o + kv4_part(c0 + p0 + c, r.item_t0, span) * E + tid;
#pragma unroll
      for (int k = 0; k < N; ++k) cp_async16(buf + c * E + tid + k * T, from + k * T, true);
    }
    if (p0 == 0)
      for (int c = tid >> 3; c < n; c += T / 8) ml[c * 8 + (tid & 7)] = __ldcg(&a.part_ml[kv4_part(c0 + c, r.item_t0, span) * 8 + (tid & 7)]);
    cp_async_wait_all();
    named_bar_sync(1, T);
    if (p0 == 0) {
#pragma unroll 1
      for (int c = 0; c < n; ++c) M = fmaxf(M, ml[c * 8 + r8].x);
    }
    const float Z = M == -INFINITY ? 0.f : M;
#pragma unroll 1
    for (int c = 0; c < np; ++c) {
      const float2 m = ml[(p0 + c) * 8 + r8];
      const float x = kv4_exp2(m.x - Z);
      L += m.y * x;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float4 u = buf[c * E + tid + k * T];
        v[k].x += x * u.x;
        v[k].y += x * u.y;
        v[k].z += x * u.z;
        v[k].w += x * u.w;
      }
    }
  }
  if (tid < 64 && l < 4) lse[r8] = kv4_lse(make_float2(M, L));
  const int row = r.row_tile * 8 + r8;
  if (row >= r.m * a.group) return;
  const float inv = L != 0.f ? 1.f / L : 0.f;
  const long to = (long)r.seq * a.out.seq + (long)(row / a.group) * a.out.row + (long)(r.head * a.group + row % a.group) * a.out.head;
#pragma unroll
  for (int k = 0; k < N; ++k)
    kv4_store4(a.out, to + (l >> 2) * (D / 8) + 4 * ((tid + k * T) >> 6), make_float4(v[k].x * inv, v[k].y * inv, v[k].z * inv, v[k].w * inv));
}
// Zeros for the query rows that no tile reaches: those of sequences without rows, and with
// zero_rest the padding.  Sequences i0, i0 + step, ..
template <int D>
__device__ __forceinline__ void kv4_zero_rows(const Kv4AttendArgs& a, const int* first, const int4* seqs, int i0, int step,
                                              int tid, int threads) {
  for (int i = i0; i < a.n_seq; i += step) {
    const int t0 = seqs[i].w > 0 ? seqs[i].z : 0, t1 = a.zero_rest ? a.q_len : seqs[i].z;  // tokens to clear
    for (int e = t0 * a.heads * (D / 4) + tid; e < t1 * a.heads * (D / 4); e += threads) {
      const int x = e % (D / 4), hq = e / (D / 4) % a.heads, tok = e / (D / 4) / a.heads;
      kv4_store4(a.out, (long)i * a.out.seq + (long)tok * a.out.row + (long)hq * a.out.head + 4 * x, make_float4(0.f, 0.f, 0.f, 0.f));
    }
  }
}

// ------------------------------------------------------------------------- the kernel
// The ring's filling, one tile at a time; called by a whole warp.
template <int D, int DT>
struct Kv4Producer {
  using O = Kv4Off<D>;
  using C = Kv4Att<D, DT>;
  Kv4Run r;
  int at, x, it, lo;
  __device__ __forceinline__ void start(int g0) {
    at = g0;
    x = it = 0;
    r.tiles = 0;
  }
  __device__ __forceinline__ bool more(int g1) const { return at + x < g1; }
  // The next tile into its stage, which is free.
  __device__ __forceinline__ void put(const Kv4AttendArgs& a, const Kv4Shared<D, DT>& sh, int g1) {
    const int lane = threadIdx.x & 31;
    if (x == r.tiles) {
      at += x;
      x = 0;
      r = kv4_run<C::kKeys>(a, sh.first, sh.seqs, at, g1);
      lo = a.window > 0 ? max(0, r.len - r.m + 1 - a.window) : 0;
    }
    const int s = it % a.stages;
    // lane b looks block b up; neighbours in the pool travel in one copy
    const int b = (r.tile + x) * C::kBlocks + lane;
    const bool want = lane < C::kBlocks && b * kKv4Block < r.len && b * kKv4Block + kKv4Block > lo;
    const long at_b = want ? kv4_block(a.c, r.slot, r.head, b) : -2;
    if (at_b == -1) set_err(a.c.err, G4_DEV_BAD_POSITION);
    const long before = __shfl_up_sync(0xFFFFFFFFu, at_b, 1);
    const uint32_t have = __ballot_sync(0xFFFFFFFFu, at_b >= 0);
    const uint32_t joins = __ballot_sync(0xFFFFFFFFu, at_b >= 0 && lane > 0 && before >= 0 && before == at_b - 1);
    if (lane == 0) {
      sh.held[s] = have;
      mbar_expect_tx(&sh.full[s], __popc(have) * O::kBlock);
    }
    __syncwarp();
    if (at_b >= 0 && !((joins >> lane) & 1)) {
      const uint32_t after = joins >> 1 >> lane;  // ones while the next block joins
      const int n = __ffs(~after);
      bulk_g2s(sh.ring + (size_t)s * C::kTile + lane * O::kBlock, a.c.data + (size_t)at_b * O::kBlock, n * O::kBlock, &sh.full[s]);
    }
    ++x;
    ++it;
  }
  // Copies in flight land before the CTA's memory goes, whatever the consumers do.
  __device__ __forceinline__ void drain(const Kv4AttendArgs& a, const Kv4Shared<D, DT>& sh) const {
    for (int k = max(0, it - a.stages); k < it; ++k) mbar_wait_drain(&sh.full[k % a.stages], (k / a.stages) & 1);
  }
};

// Returns the first tile of the last run.
template <int D, int DT, bool WIDE>
__device__ __forceinline__ int kv4_consume(const Kv4AttendArgs& a, const Kv4Shared<D, DT>& sh, int g0, int g1) {
  using O = Kv4Off<D>;
  using C = Kv4Att<D, DT>;
  constexpr int W = D / 32, NB = C::kNB;  // words of a key (or value pair) per lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int set = warp >> 2, wq = warp & 3;
  const float score_scale = WIDE ? a.scale : a.scale * kKv4Up;
  Kv4Producer<D, DT> fill;
  if (!C::kOwnProducer) {
    fill.start(g0);
    if (warp == 0)
      while (fill.it < a.stages && fill.more(g1)) fill.put(a, sh, g1);
  }
  int it = 0, piece = 0, last_at = g0;
  for (int at = g0; at < g1; ++piece) {
    const Kv4Run r = kv4_run<C::kKeys>(a, sh.first, sh.seqs, at, g1);
    const int n_rows = r.m * a.group, row0 = r.row_tile * 8;
    named_bar_sync(1, 32 * C::kWarps);
    kv4_stage_q<D, DT>(a, sh.qs, r.seq, r.head, row0, n_rows, threadIdx.x, 32 * C::kWarps);
    named_bar_sync(1, 32 * C::kWarps);

    float acc[D / 16][4];
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    float mx0 = -INFINITY, mx1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    // rows that query rows 2t and 2t + 1 see: (low, last]
    const int ra = min(row0 + 2 * t, n_rows - 1), rb = min(row0 + 2 * t + 1, n_rows - 1);
    const int last0 = r.len - r.m + ra / a.group, last1 = r.len - r.m + rb / a.group;
    const int low0 = a.window > 0 ? last0 - a.window : -1, low1 = a.window > 0 ? last1 - a.window : -1;
    const int last_min = r.len - r.m + min(row0, n_rows - 1) / a.group;
    const int low_max = a.window > 0 ? r.len - r.m + min(row0 + 7, n_rows - 1) / a.group - a.window : -1;

    for (int x = 0; x < r.tiles; ++x, ++it) {
      if (!C::kOwnProducer && warp == 0) {
        // stages that their warps have left are filled again; only the tile at hand is waited for
        while (fill.more(g1) && !__any_sync(0xFFFFFFFFu, *sh.abort_flag)) {
          if (fill.it >= a.stages) {
            uint64_t* e = &sh.empty[fill.it % a.stages];
            const uint32_t parity = (fill.it / a.stages - 1) & 1;
            bool free_now = __all_sync(0xFFFFFFFFu, mbar_try(e, parity));
            if (!free_now && fill.it <= it) free_now = kv4_wait_warp(e, parity, sh.abort_flag);
            if (!free_now) break;
          }
          fill.put(a, sh, g1);
        }
      }
      if (C::kSets > 1 && it % C::kSets != set) continue;
      const int s = it % a.stages;
      const bool here = kv4_wait_warp(&sh.full[s], (it / a.stages) & 1, sh.abort_flag);
      const uint32_t have = here ? sh.held[s] >> (wq * C::kBpw) & ((1u << C::kBpw) - 1u) : 0u;
      if (have) {
        // the warp's blocks of the tile are neighbours: 16 NB consecutive keys
        const uint8_t* blk = sh.ring + (size_t)s * C::kTile + wq * C::kBpw * O::kBlock;
        const int j0 = ((r.tile + x) * C::kBlocks + wq * C::kBpw) * kKv4Block;
        float c[NB][4];
        kv4_scores<D, C::kQP, NB, WIDE>(
            sh.qs, lane, [&](int b, int i) { return reinterpret_cast<const uint4*>(blk + b * O::kBlock)[i * 32 + lane]; },
            [&](int b, int half) { return kv4_key_scales<D>(blk + b * O::kBlock + O::kKs, g + 8 * half, t); }, c);
        float n0 = -INFINITY, n1 = -INFINITY;
        const bool edge = have != (1u << C::kBpw) - 1u || j0 + 16 * NB - 1 > last_min || j0 <= low_max;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
          for (int j = 0; j < 4; ++j) c[b][j] = __fmul_rn(c[b][j], score_scale);  // keys g (0, 1) and g + 8 (2, 3); rows 2t, 2t + 1
          if (edge) {
            const int ja = j0 + 16 * b + g, jb = ja + 8;
            const bool gone = !((have >> b) & 1);  // no page, or wholly outside: whatever the ring holds there
            if (gone || ja > last0 || ja <= low0) c[b][0] = -INFINITY;
            if (gone || ja > last1 || ja <= low1) c[b][1] = -INFINITY;
            if (gone || jb > last0 || jb <= low0) c[b][2] = -INFINITY;
            if (gone || jb > last1 || jb <= low1) c[b][3] = -INFINITY;
          }
          n0 = fmaxf(n0, fmaxf(c[b][0], c[b][2]));
          n1 = fmaxf(n1, fmaxf(c[b][1], c[b][3]));
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          n0 = fmaxf(n0, __shfl_xor_sync(0xFFFFFFFFu, n0, o));
          n1 = fmaxf(n1, __shfl_xor_sync(0xFFFFFFFFu, n1, o));
        }
        if (__any_sync(0xFFFFFFFFu, n0 > mx0 || n1 > mx1)) {
          n0 = fmaxf(n0, mx0);
          n1 = fmaxf(n1, mx1);
          // a row that has seen nothing yet keeps -inf and sums of zero
          const float f0 = n0 == -INFINITY ? 1.f : kv4_exp2(mx0 - n0), f1 = n1 == -INFINITY ? 1.f : kv4_exp2(mx1 - n1);
          mx0 = n0;
          mx1 = n1;
          l0 *= f0;
          l1 *= f1;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            acc[i][0] *= f0;
            acc[i][1] *= f1;
            acc[i][2] *= f0;
            acc[i][3] *= f1;
          }
        }
        const float z0 = mx0 == -INFINITY ? 0.f : mx0, z1 = mx1 == -INFINITY ? 0.f : mx1;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (edge && !((have >> b) & 1)) continue;  // its codes may be anything: not even times zero
          const float p00 = kv4_exp2(c[b][0] - z0), p01 = kv4_exp2(c[b][1] - z1);
          const float p10 = kv4_exp2(c[b][2] - z0), p11 = kv4_exp2(c[b][3] - z1);
          l0 += p00 + p10;
          l1 += p01 + p11;
          uint32_t pa[C::kPP], pb[C::kPP];
          kv4_split<C::kPP>(p00, p01, pa);
          kv4_split<C::kPP>(p10, p11, pb);
#pragma unroll
          for (int part = 0; part < C::kPP; ++part) {
            pa[part] = kv4_transpose(pa[part]);
            pb[part] = kv4_transpose(pb[part]);
          }
          // output: 16 numbers of the values (rows of the product) by 8 query rows, over 16 keys
          const uint4* vc = reinterpret_cast<const uint4*>(blk + b * O::kBlock + O::kV) + lane;
          const uint32_t* vs = reinterpret_cast<const uint32_t*>(blk + b * O::kBlock + O::kVs);
          constexpr int G = D > 256 ? D / 256 : 1;  // groups among a lane's D / 8 numbers
#pragma unroll
          for (int k = 0; k < G; ++k) {
            const int grp = D >= 256 ? g * G + k : g * D / 256;
            const Kv4Scale<WIDE> sa(vs[grp * 8 + t]), sb(vs[grp * 8 + t + 4]);
#pragma unroll
            for (int i = k * (W / 2 / G); i < (k + 1) * (W / 2 / G); ++i) {
              const uint4 u = vc[i * 32];  // row pair t: words 2i, 2i + 1; pair t + 4: same
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t ua = e ? u.y : u.x, ub = e ? u.w : u.z;
                const uint32_t a0 = sa.template pair<0>(ua), a1 = sa.template pair<1>(ua), a2 = sb.template pair<0>(ub), a3 = sb.template pair<1>(ub);
                const uint32_t b0 = sa.template pair<2>(ua), b1 = sa.template pair<3>(ua), b2 = sb.template pair<2>(ub), b3 = sb.template pair<3>(ub);
#pragma unroll
                for (int part = 0; part < C::kPP; ++part) {
                  kv4_mma(acc[4 * i + 2 * e], a0, a1, a2, a3, pa[part], pb[part]);
                  kv4_mma(acc[4 * i + 2 * e + 1], b0, b1, b2, b3, pa[part], pb[part]);
                }
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[s]);
    }
    at += r.tiles;

    // ---- join the warps' sums
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, o);
      l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, o);
    }
    if (g == 0) {
      sh.mls[warp * 8 + 2 * t] = make_float2(mx0, l0);
      sh.mls[warp * 8 + 2 * t + 1] = make_float2(mx1, l1);
    }
    named_bar_sync(1, 32 * C::kWarps);
    float M0 = -INFINITY, M1 = -INFINITY, L0 = 0.f, L1 = 0.f;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) {
      M0 = fmaxf(M0, sh.mls[w * 8 + 2 * t].x);
      M1 = fmaxf(M1, sh.mls[w * 8 + 2 * t + 1].x);
    }
    const float Z0 = M0 == -INFINITY ? 0.f : M0, Z1 = M1 == -INFINITY ? 0.f : M1;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) {
      const float2 u = sh.mls[w * 8 + 2 * t], v = sh.mls[w * 8 + 2 * t + 1];
      L0 += u.y * kv4_exp2(u.x - Z0);
      L1 += v.y * kv4_exp2(v.x - Z1);
    }
    const bool whole = r.whole;
    // a whole item is divided by its sum here, a partial one when the spans are joined
    const float up = WIDE ? 1.f : kKv4Up;
    const float f0 = kv4_exp2(mx0 - Z0) * up * (whole ? (L0 != 0.f ? 1.f / L0 : 0.f) : 1.f);
    const float f1 = kv4_exp2(mx1 - Z1) * up * (whole ? (L1 != 0.f ? 1.f / L1 : 0.f) : 1.f);
    auto put = [&](bool add) {
#pragma unroll
      for (int w = 0; w < W; ++w)
#pragma unroll
        for (int sel = 0; sel < 2; ++sel) {
          const float f = sel ? f1 : f0;
          float4* p = &sh.os[(((warp % C::kRegions) * W + w) * 2 + sel) * 32 + lane];
          float4 v = make_float4(acc[2 * w][sel] * f, acc[2 * w][2 + sel] * f, acc[2 * w + 1][sel] * f, acc[2 * w + 1][2 + sel] * f);
          if (add) {
            const float4 u = *p;
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
          }
          *p = v;
        }
    };
#pragma unroll
    for (int round = C::kWarps / C::kRegions - 1; round >= 0; --round) {
      if (warp / C::kRegions == round) put(round + 1 < C::kWarps / C::kRegions);
      named_bar_sync(1, 32 * C::kWarps);
    }
    const long slot_p = (long)blockIdx.x * 2 + (piece ? 1 : 0);
    // entry e: lane l of word w: numbers (l / 4) D/8 + 4w .. of query row 2 (l % 4) + sel
    for (int e = threadIdx.x; e < W * 64; e += 32 * C::kWarps) {
      const int l = e & 31, sel = (e >> 5) & 1, w = e >> 6;
      float4 v = sh.os[e];
#pragma unroll
      for (int k = 1; k < C::kRegions; ++k) {
        const float4 u = sh.os[k * W * 64 + e];
        v.x += u.x;
        v.y += u.y;
        v.z += u.z;
        v.w += u.w;
      }
      if (!whole) {
        a.part_o[slot_p * W * 64 + e] = v;
      } else {
        const int row = row0 + 2 * (l & 3) + sel;
        if (row < n_rows) {
          const int tok = row / a.group, hq = r.head * a.group + row % a.group;
          kv4_store4(a.out, (long)r.seq * a.out.seq + (long)tok * a.out.row + (long)hq * a.out.head + (l >> 2) * (D / 8) + 4 * w, v);
        }
      }
    }
    if (threadIdx.x < 32 && g == 0) {
      if (!whole) {
        a.part_ml[slot_p * 8 + 2 * t] = make_float2(M0, L0);
        a.part_ml[slot_p * 8 + 2 * t + 1] = make_float2(M1, L1);
      } else {
        float* lse = a.lse + ((long)r.seq * a.c.kvh + r.head) * a.lse_rows + r.row_tile * 8 + 2 * t;
        lse[0] = L0 != 0.f ? M0 + log2f(L0) : INFINITY;
        lse[1] = L1 != 0.f ? M1 + log2f(L1) : INFINITY;
      }
    }
    last_at = at - r.tiles;
  }
  if (!C::kOwnProducer && warp == 0) fill.drain(a, sh);
  if (*sh.abort_flag && threadIdx.x == 0) set_err(a.c.err, G4_DEV_TIMEOUT);
  return last_at;
}

// The shared items that a CTA's span begins and ends with: the CTA that finishes its part of an
// item last joins all of them.  After the span, so that nothing of it weighs on the loop's
// registers.
template <int D, int DT>
__device__ __forceinline__ void kv4_join_span(const Kv4AttendArgs& a, const Kv4Shared<D, DT>& sh, int g0, int g1, int last_at, int span) {
  using C = Kv4Att<D, DT>;
  if (g0 >= g1) return;
  __threadfence();
#pragma unroll 1
  for (int k = 0; k < (last_at > g0 ? 2 : 1); ++k) {
    const Kv4Run r = kv4_run<C::kKeys>(a, sh.first, sh.seqs, k ? last_at : g0, g1);
    if (r.whole) continue;
    const int c0 = (unsigned)r.item_t0 / (unsigned)span, c1 = (unsigned)(r.item_t0 + r.of - 1) / (unsigned)span;
    const long item = ((long)r.seq * a.c.kvh + r.head) * a.row_tiles + r.row_tile;
    named_bar_sync(1, 32 * C::kWarps);  // every thread's sums are out
    if (threadIdx.x == 0) {
      const bool is_last = atomicAdd(a.tickets + item, 1u) == (unsigned)(c1 - c0);
      if (is_last) a.tickets[item] = 0;
      *sh.last = is_last;
    }
    named_bar_sync(1, 32 * C::kWarps);
    if (!*sh.last) continue;
    __threadfence();
    kv4_join_ring<D, DT>(a, sh, r, span, c0, c1, a.lse + item * 8);
  }
}

template <int D, int DT>
__global__ void __launch_bounds__(Kv4Att<D, DT>::kThreads, Kv4Att<D, DT>::kMinCtas) kv4_attend_kernel(const __grid_constant__ Kv4AttendArgs a) {
  using O = Kv4Off<D>;
  using C = Kv4Att<D, DT>;
  extern __shared__ __align__(128) uint8_t kv4_smem[];
  const Kv4Shared<D, DT> sh(kv4_smem, a.stages, a.n_seq);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 4);
    }
    *sh.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();
  const int wide = __ldcg(a.c.wide) | a.plain;
  kv4_plan<C::kKeys>(a, sh.first, sh.seqs, reinterpret_cast<int*>(sh.os), blockIdx.x == 0);
  const int total = sh.first[a.n_seq];
  const int span = kv4_span(a, sh.first, gridDim.x);
  const int g0 = (int)min((unsigned)total, blockIdx.x * (unsigned)span), g1 = (int)min((unsigned)total, (unsigned)g0 + span);
  if (warp < C::kWarps) {
    const int last_at = wide ? kv4_consume<D, DT, true>(a, sh, g0, g1) : kv4_consume<D, DT, false>(a, sh, g0, g1);
    if (a.join_inside) {
      kv4_join_span<D, DT>(a, sh, g0, g1, last_at, span);
      kv4_zero_rows<D>(a, sh.first, sh.seqs, blockIdx.x, gridDim.x, threadIdx.x, 32 * C::kWarps);
    }
    return;
  }
  // ---- producer: tiles into the ring
  Kv4Producer<D, DT> fill;
  fill.start(g0);
  while (fill.more(g1)) {
    const int s = fill.it % a.stages;
    if (fill.it >= a.stages && !kv4_wait_warp(&sh.empty[s], (fill.it / a.stages - 1) & 1, sh.abort_flag)) {
      if (lane == 0) set_err(a.c.err, G4_DEV_TIMEOUT);
      break;
    }
    fill.put(a, sh, g1);
  }
  fill.drain(a, sh);
}

// -------------------------------------------------------------------------- the finish
// Second launch.  CTAs with blockIdx.y < join_ctas (none when the first launch joins inside) add
// the partial sums that the spans left of item blockIdx.x, in span order, each a share of its
// numbers.  With an account and one item per (sequence, KV head), the others each
// take a run of the item's keys and add the weights those received, p = 2^(s - lse), recomputed
// from the keys: a score per key and query row kept from the first launch would cost 64 bytes of
// traffic a key and a buffer of its own, the codes cost 9/16 D and are still in L2 for the most.
constexpr int kKv4FinishThreads = 128;

// Adds what the keys `key` and key + 8 of a block receive from eight query rows (this lane: rows
// 2t and 2t + 1), given the log2 of each row's softmax sum.
template <int D, int DT, bool WIDE>
__device__ __forceinline__ void kv4_gain_tile(const Kv4AttendArgs& a, const uint4* qs, const uint8_t* blk, int lane,
                                              const uint4 (&u)[D / 64], const Kv4KeyScales<D>& s0, const Kv4KeyScales<D>& s1,
                                              int key, const float* lse8, int len, int m, int row0, int n_rows,
                                              float& gain0, float& gain1) {
  const int t = lane & 3;
  float c[1][4];
  kv4_scores<D, Kv4Att<D, DT>::kQP, 1, WIDE>(qs, lane, [&](int, int i) { return u[i]; },
                                             [&](int, int half) { return half ? s1 : s0; }, c);
  const float sc = WIDE ? a.scale : a.scale * kKv4Up, e0 = lse8[2 * t], e1 = lse8[2 * t + 1];
  const int ra = row0 + 2 * t, rb = ra + 1;
  const int last0 = ra < n_rows ? len - m + ra / a.group : -1, last1 = rb < n_rows ? len - m + rb / a.group : -1;
  if (key <= last0) gain0 += kv4_exp2(__fmul_rn(c[0][0], sc) - e0);
  if (key <= last1) gain0 += kv4_exp2(__fmul_rn(c[0][1], sc) - e1);
  if (key + 8 <= last0) gain1 += kv4_exp2(__fmul_rn(c[0][2], sc) - e0);
  if (key + 8 <= last1) gain1 += kv4_exp2(__fmul_rn(c[0][3], sc) - e1);
}
// A block's codes and scales of this lane, from global memory.
template <int D>
struct Kv4KeyBlock {
  uint4 u[D / 64];
  Kv4KeyScales<D> s0, s1;
  __device__ __forceinline__ void load(const uint8_t* blk, int lane) {
    using O = Kv4Off<D>;
#pragma unroll
    for (int k = 0; k < D / 64; ++k) u[k] = __ldcg(reinterpret_cast<const uint4*>(blk) + k * 32 + lane);
    s0 = kv4_key_scales<D>(blk + O::kKs, lane >> 2, lane & 3);
    s1 = kv4_key_scales<D>(blk + O::kKs, (lane >> 2) + 8, lane & 3);
  }
};
// Adds the gains of keys g and g + 8 of block b (pool index at) to the account.
__device__ __forceinline__ void kv4_add_gain(const Kv4AttendArgs& a, long at, int b, int len, int lane, float gain0, float gain1) {
  gain0 += __shfl_xor_sync(0xFFFFFFFFu, gain0, 1);
  gain1 += __shfl_xor_sync(0xFFFFFFFFu, gain1, 1);
  gain0 += __shfl_xor_sync(0xFFFFFFFFu, gain0, 2);
  gain1 += __shfl_xor_sync(0xFFFFFFFFu, gain1, 2);
  const int g = lane >> 2, t = lane & 3;
  if (t < 2 && b * kKv4Block + g + 8 * t < len) a.c.weight[at * kKv4Block + g + 8 * t] += t ? gain1 : gain0;
}

template <int D, int DT>
__global__ void __launch_bounds__(kKv4FinishThreads) kv4_finish_kernel(const __grid_constant__ Kv4AttendArgs a, int ctas, int join_ctas) {
  using C = Kv4Att<D, DT>;
  using O = Kv4Off<D>;
  extern __shared__ __align__(128) uint8_t kv4_smem[];
  int4* seqs = reinterpret_cast<int4*>(kv4_smem);
  uint4* qs = reinterpret_cast<uint4*>(seqs + a.n_seq);
  int* first = reinterpret_cast<int*>(qs + C::kQBytes / 16);
  __shared__ float2 ml[8 + 8 * kKv4FinishThreads / 32];
  __shared__ float sE[8];
  const int item = blockIdx.x, per_seq = a.c.kvh * a.row_tiles, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i = item / per_seq, x = item % per_seq, head = x / a.row_tiles, rt = x % a.row_tiles;
  const bool join = (int)blockIdx.y < join_ctas;
  // What the first launch reads as well can be read before it has ended.
  const int wide = __ldcg(a.c.wide) | a.plain;
  kv4_plan<C::kKeys>(a, first, seqs, first + a.n_seq + 2, false);
  const int slot = seqs[i].x, len = seqs[i].y, m = seqs[i].z, n = seqs[i].w, n_rows = m * a.group;
  if (!join && n > 0) kv4_stage_q<D, DT>(a, qs, i, head, 0, n_rows, tid, kKv4FinishThreads);
  const int span = kv4_span(a, first, ctas);
  const int t0 = first[i] + n * x;  // the item's first tile
  const int c0 = (unsigned)t0 / (unsigned)span, c1 = n ? (int)((unsigned)(t0 + n - 1) / (unsigned)span) : c0 - 1;
  pdl_wait();
  pdl_trigger();
  if (join) {
    if (x == 0 && blockIdx.y == 0) kv4_zero_rows<D>(a, first, seqs, i, a.n_seq, tid, kKv4FinishThreads);
    if (c1 <= c0) return;  // nothing to see, or one CTA had the whole item
  } else if (n == 0) {
    return;
  }
  if (c0 < c1 && !a.join_inside) {
    kv4_join_ml(a, t0, span, c0, c1, tid, kKv4FinishThreads / 32, ml, 1);
    if (tid < 8) {
      sE[tid] = kv4_lse(ml[tid]);
      if (blockIdx.y == 0) a.lse[(long)item * 8 + tid] = sE[tid];
    }
  } else if (tid < 8) {
    sE[tid] = __ldcg(a.lse + (long)item * 8 + tid);
  }
  __syncthreads();
  if (join) {
    kv4_join_rows<D>(a, i, head, rt * 8, n_rows, t0, span, c0, c1, ml, blockIdx.y * kKv4FinishThreads + tid,
                     join_ctas * kKv4FinishThreads);
    return;
  }
  // ---- the account of a run of keys (row_tiles == 1)
  const int nb = (len + kKv4Block - 1) / kKv4Block, step = (gridDim.y - join_ctas) * 4;
  for (int b = (blockIdx.y - join_ctas) * 4 + warp; b < nb; b += step) {
    const long at = kv4_block(a.c, slot, head, b);
    if (at < 0) continue;
    const uint8_t* blk = a.c.data + (size_t)at * O::kBlock;
    Kv4KeyBlock<D> kb;
    kb.load(blk, lane);
    float gain0 = 0.f, gain1 = 0.f;
    const int key = b * kKv4Block + (lane >> 2);
    if (wide) kv4_gain_tile<D, DT, true>(a, qs, blk, lane, kb.u, kb.s0, kb.s1, key, sE, len, m, 0, n_rows, gain0, gain1);
    else kv4_gain_tile<D, DT, false>(a, qs, blk, lane, kb.u, kb.s0, kb.s1, key, sE, len, m, 0, n_rows, gain0, gain1);
    kv4_add_gain(a, at, b, len, lane, gain0, gain1);
  }
}

// ------------------------------------------------------------------------- the account
// Blocks of query tokens (more than eight query rows per KV head): a warp holds 16 keys of one
// (sequence, KV head) in registers and takes every query row past them, eight at a time, so a
// row's gain is one warp's sum in a fixed order.  28 query rows over five sequences of 1,531 rows, four
// KV heads of 64: 9 us, bound by latency (about two warps a scheduler).
constexpr int kKv4GainWarps = 4;

template <int D, int DT>
__global__ void __launch_bounds__(32 * kKv4GainWarps) kv4_gain_kernel(const __grid_constant__ Kv4AttendArgs a) {
  using O = Kv4Off<D>;
  extern __shared__ __align__(128) uint8_t kv4_smem[];
  uint4* qs = reinterpret_cast<uint4*>(kv4_smem);
  __shared__ float lse8[8];
  const int i = blockIdx.y, h = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
  pdl_wait();
  pdl_trigger();
  int slot, len, m;
  if (!kv4_seq(a, i, &slot, &len, &m) || m == 0) return;
  if (kv4_repeated(a.slots, i, slot)) return;
  const int wide = __ldcg(a.c.wide) | a.plain;
  const int n_rows = m * a.group;
  const int nb = (len + kKv4Block - 1) / kKv4Block;
  for (int b0 = blockIdx.x * kKv4GainWarps; b0 < nb; b0 += gridDim.x * kKv4GainWarps) {
    const int b = b0 + warp;
    const long at = b < nb ? kv4_block(a.c, slot, h, b) : -1;
    const uint8_t* blk = a.c.data + (size_t)(at < 0 ? 0 : at) * O::kBlock;
    Kv4KeyBlock<D> kb;
    kb.load(blk, lane);
    float gain0 = 0.f, gain1 = 0.f;  // keys g and g + 8
    // the first row tile that any key of the CTA is seen by
    const int tok0 = max(0, b0 * kKv4Block - (len - m));
    for (int rt = tok0 * a.group / 8; rt * 8 < n_rows; ++rt) {
      __syncthreads();
      kv4_stage_q<D, DT>(a, qs, i, h, rt * 8, n_rows, threadIdx.x, 32 * kKv4GainWarps);
      if (threadIdx.x < 8) lse8[threadIdx.x] = __ldcg(a.lse + ((long)i * a.c.kvh + h) * a.lse_rows + rt * 8 + threadIdx.x);
      __syncthreads();
      if (at < 0) continue;
      if (wide) kv4_gain_tile<D, DT, true>(a, qs, blk, lane, kb.u, kb.s0, kb.s1, b * kKv4Block + g, lse8, len, m, rt * 8, n_rows, gain0, gain1);
      else kv4_gain_tile<D, DT, false>(a, qs, blk, lane, kb.u, kb.s0, kb.s1, b * kKv4Block + g, lse8, len, m, rt * 8, n_rows, gain0, gain1);
    }
    if (at >= 0) kv4_add_gain(a, at, b, len, lane, gain0, gain1);
  }
}

}  // namespace g4
