// Attention over 16-bit keys and values on the 5th-generation tensor cores: whole prompts (causal,
// packed sequences, optionally a sliding window), and the part of a batch's tokens over a prefix that
// all its sequences share.
//
//   s_j = scale * q . K_j     p_j = 2^(s_j log2 e - m)     o = sum p_j V_j / sum p_j
//
// The query rows of a KV head are its tokens' heads, token after token (row t * G + g): a block is as
// many whole tokens as the 128 rows of a product hold.  A CTA takes items of NQ blocks past tiles of
// 128 keys:
//   one warp copies an item's queries, and tiles of keys and values into a ring of 128-byte-swizzled
//   stages, by TMA,
//   a warp issues S = Q K^T (both operands shared, fp32 in tensor memory) and O += P V (P in
//   tensor memory, in the columns of the S that it was made of),
//   four warps for each block of rows take a row per thread: maximum, exponentials, sum; with NQ 1 four
//   more give out an item's results while the next item's weights are made.
// With heads up to 128 two blocks of rows share each tile (NQ 2): while one's weights are made, the
// other's products run.  Wider heads leave room for one block's output (256 columns of the 512); its
// scores then have two buffers, and the next tile's product runs while a tile's weights are made.
// 512-wide heads take two items per block of rows, each with half of the values' columns and scores of
// its own: half as many products again, where the whole output would leave no column for scores.
//
// A row's reference m is raised, and its output so far rescaled, only when a score exceeds it by 2^8:
// weights up to 256 lose nothing in fp32, nor in P.  P is rounded to the values' 16-bit type (the
// operands of a product have one type): each weight is off by at most 2^-8 of itself (bf16; fp16:
// 2^-11, and weights below 2^-20 by up to 2^-31), independently of the others, while the sum that
// divides them is of the unrounded ones.
//
// Measured (bf16 unless said; useful operations, the triangle's half of the tiles at its edge not counted):
//   16,384 tokens, 32 heads on 8 of 128         1,360 us, 1.62 PFLOP/s; tensor pipe busy 73%: two chains of scores ->
//     maximum, exponentials (1,250 cycles a tile) -> product share it, and the operands' bytes in shared memory
//     take as long as the products (a tile of both blocks: 2,048 cycles of either, 2,480 measured)
//   8 prompts of 2,250 to 4,000, 8 heads on 1 of 512   660 us, 1.00 PFLOP/s (1.50 with the scores made twice); busy 69%: a
//     ring of three stages waits for L2 a sixth of the time
//   the same of 256, window 512                 103 us, 0.93 PFLOP/s; busy 47%: items of five tiles, whose first scores
//     and last product nothing else covers
//   61 prompts of 168 to 333, 12 heads on 4 of 64 (fp16)   40 us; items of one to three tiles: latency of their chains
//   one of 128 tokens, 8 heads on 1 of 256      9.2 us: latency of one tile's chain
#pragma once
#include <cuda.h>

#include <cstddef>

#include "tc05.cuh"

namespace g4 {

constexpr int kAttM = 128;  // query rows of a block
constexpr int kAttN = 128;  // keys of a tile

template <int D>
struct Att16 {
  static constexpr int NQ = D <= 128 ? 2 : 1;
  static constexpr int DV = D == 512 ? 256 : D;           // values' columns of an item
  static constexpr int HV = D / DV;                       // items of a block of rows
  static constexpr int kSlab = kAttN * 128;               // 128 rows of 64 numbers
  static constexpr int kStage = D == 64 ? kSlab : 2 * kSlab;
  static constexpr int KS = D * 2 * kAttN / kStage;       // stages of a tile of keys, by their columns
  static constexpr int VS = DV * 2 * kAttN / kStage;      // and of values, by their rows
  static constexpr int kVRows = kAttN / VS;               // rows of a stage of values
  static constexpr int kStages = D == 64 ? 8 : D == 512 ? 3 : 5;
  static constexpr int kQ = NQ * kAttM * D * 2;
  static constexpr int kSoftWarps = 4 * NQ;
  static constexpr int kThreads = 384;                    // softmax, four other warps, NQ 1: four that give out results
  static constexpr int kColS = NQ * DV;                   // tensor memory: outputs, then two buffers of scores
  static constexpr size_t kSmem = 1024 + kQ + (size_t)kStages * kStage + 512 + (NQ == 1 ? kAttM * 4 : 0);
};

struct Att16Item {
  int row0;       // first packed row of the sequence; below 0: no item is left, and lo .. hi - 1 are the rows that all span
  int t0, len;    // first token of the item; tokens of the sequence
  int head, half;
  int lo, hi;     // keys lo .. hi - 1 of the sequence
  int part;       // prefix: slot of its partial result
};

// Whether an item's last tile reaches past the sequence (PREFIX: the prefix), where anything may lie: the next
// sequence's rows, or what a program left behind the last.  So can the tile of an item that ends before its sequence does.
template <bool PREFIX>
__device__ __forceinline__ bool att_past_end(const Att16Item& it) {
  const int tiles = (it.hi - it.lo + kAttN - 1) / kAttN;
  return it.lo + tiles * kAttN > (PREFIX ? it.hi : it.len);
}

struct Att16Bars {
  uint64_t full[8];
  uint64_t empty[8], sfull[2], pvdone[2], qdone, odone;  // what commits arrive at, in this order (the end of the warp that issues)
  uint64_t pfull[2], qfull, ifull[2], iempty[2], vneed, vtail, lfull, ofree, drained;
  Att16Item item[2];
  uint32_t tmem;
  int abort;
  int beat;  // steps of att_repair
};
static_assert(sizeof(Att16Bars) <= 512, "barriers");
static_assert(offsetof(Att16Bars, sfull) == 8 * 16 && offsetof(Att16Bars, odone) == 8 * 21, "the order of the barriers");

struct Att16Args {
  const uint16_t* q;
  uint16_t* out;
  const uint16_t* v;  // prompt: for rows whose unseen keys carry values that are not finite
  const uint16_t* k;
  long q_row, q_head, o_row, o_head, k_row, k_head, v_row, v_head;  // strides in elements
  int o_vec;          // accesses of 16 bytes (1) or 32 (2)
  int group, kvh;
  int tb;             // tokens of a block: kAttM / group
  float scale;        // times log2 e
  int* err;
  // prompt
  const int* offsets;  // [n_seq + 1]
  int n_seq, n_rows, window;
  int zero_rest;       // rows in front of the first sequence and behind the last become zeros
  unsigned* ticket;    // [2]: the next item, CTAs that are done
  // prefix
  const int *table, *slots, *lens;
  int n_slots, n_pages, log_page, max_pages;
  int keys, splits, tiles_per;  // keys of the prefix; parts of a block of rows, of tiles_per tiles each
  float* part_o;       // [part][NQ * 128 rows][D]
  float2* part_ml;     // [part][NQ * 128 rows]
};

__device__ __forceinline__ float att_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float att_max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Two fp32 numbers at a time.
__device__ __forceinline__ uint64_t att_two(float lo, float hi) {
  uint64_t y;
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(lo), "f"(hi));
  return y;
}
__device__ __forceinline__ uint64_t att_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t y;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
  return y;
}
__device__ __forceinline__ uint64_t att_mul2(uint64_t a, uint64_t b) {
  uint64_t y;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
  return y;
}
__device__ __forceinline__ uint64_t att_add2(uint64_t a, uint64_t b) {
  uint64_t y;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
  return y;
}
__device__ __forceinline__ void att_split(uint64_t x, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x)); }
// 32 bytes to a 32-byte-aligned address: a whole sector at a time.
__device__ __forceinline__ void att_store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
               "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// Two numbers rounded to the 16-bit type (BF: bf16, else fp16), the first in the low half.
template <bool BF>
__device__ __forceinline__ uint32_t att_pack(float lo, float hi) {
  uint32_t r;
  if (BF) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Number x of eight.
template <bool BF>
__device__ __forceinline__ float att_one(const uint4& v, int x) {
  const uint32_t w = x < 2 ? v.x : x < 4 ? v.y : x < 6 ? v.z : v.w;
  if (BF) return __uint_as_float(x & 1 ? w & 0xFFFF0000u : w << 16);
  const uint16_t u = (uint16_t)(x & 1 ? w >> 16 : w);
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(u));
  return f;
}
// Weights go into products times 2^this: fp16 ones reach up to 2^8 . 2^6, and lose bits from 2^-20 down instead of 2^-14.
template <bool BF>
__device__ __forceinline__ constexpr float att_up() { return BF ? 0.f : 6.f; }
__device__ __forceinline__ bool att_finite(float x) { return fabsf(x) < INFINITY; }

// kind::f16: operands of the type, fp32 result, M 128.
template <bool BF>
__device__ __forceinline__ constexpr uint32_t att_idesc(int n, bool b_leading) {
  return (1u << 4) | (BF ? (1u << 7) | (1u << 10) : 0u) | (b_leading ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kAttM >> 4) << 24);
}
// A descriptor `bytes` further into shared memory (its address field does not carry into the next one).
__device__ __forceinline__ uint64_t att_desc_at(uint64_t desc, uint32_t bytes) {
  return (desc & 0xFFFFFFFF00000000ull) | (uint32_t)((uint32_t)desc + (bytes >> 4));
}
// The warp that issues matrix instructions walks through its loops as one, so that what it computes is the
// same in all lanes and descriptors come from uniform registers; the thread with `one` issues.  (Inside a
// branch that one thread takes, each product cost some 80 cycles to issue, more than its 64 in the
// pipe: 16,384 tokens took 1,630 us instead of 1,325.)
__device__ __forceinline__ uint32_t att_elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p;
}
__device__ __forceinline__ void att_commit(uint32_t one, uint64_t* b) {
  asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(su32(b)), "r"(one) : "memory");
}
__device__ __forceinline__ void att_mma_ts(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc), "r"(one) : "memory");
}
__device__ __forceinline__ void att_mma_ss(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc), "r"(one) : "memory");
}
__device__ __forceinline__ void att_tma3(void* dst, const CUtensorMap* m, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(su32(dst)),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(su32(bar))
      : "memory");
}
// The same of rank 4, and the barrier's count of its bytes, by the thread with `one`.
__device__ __forceinline__ void att_tma4(uint32_t one, void* dst, const CUtensorMap* m, int x, int y, int z, int w, uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %8, 0;\n @q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%6], %7;\n"
      " @q cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n}\n" ::"r"(su32(dst)),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(w), "r"(su32(bar)), "r"(bytes), "r"(one)
      : "memory");
}
__device__ __forceinline__ void att_tma2(void* dst, const CUtensorMap* m, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(su32(dst)),
      "l"(m), "r"(x), "r"(y), "r"(su32(bar))
      : "memory");
}
// Waits until nothing has gone on for two seconds: a CTA whose rows are made anew (att_repair) may take longer for an item, and
// counts its steps.  False when the time is up, or was for another thread of the CTA.
__device__ __forceinline__ bool att_wait(uint64_t* b, uint32_t parity, Att16Bars* s) {
  if (mbar_try(b, parity)) return true;
  volatile int* const abort = reinterpret_cast<volatile int*>(&s->abort);
  volatile int* const beat = reinterpret_cast<volatile int*>(&s->beat);
  uint64_t now, end = 0;
  int seen = 0;
  while (!*abort) {
    for (int i = 0; i < 256; ++i)
      if (mbar_try(b, parity)) return true;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(now));
    const int steps = *beat;
    if (end == 0 || steps != seen) {
      end = now + 2000000000ull;
      seen = steps;
    } else if (now > end) {
      *abort = 1;
    }
  }
  return false;
}

// The issuing warp's last wait.  Nothing says that commits arrive in the order in which they were made, so the last arrival at
// each of their barriers is waited for, also behind a wait that gave up; every earlier one has been waited for by the role
// that it is for.  A lane takes a barrier; the numbers are those of its commits (the ring's stages: `lap` each, one more for
// the first `st`).  (A call: written out in its place it cost the long prompts 1% by where the rest came to lie.)
__device__ __noinline__ void att_last(Att16Bars* s, int stages, int st, int lap, int sfull0, int sfull1, int pvdone0, int pvdone1, int qdone,
                                      int odone) {
  const int lane = threadIdx.x & 31;
  int commits = lane < stages ? lap + (lane < st) : 0;
  if (lane >= 8 && lane < 10) commits = lane & 1 ? sfull1 : sfull0;
  if (lane >= 10 && lane < 12) commits = lane & 1 ? pvdone1 : pvdone0;
  if (lane == 12) commits = qdone;
  if (lane == 13) commits = odone;
  if (commits > 0) mbar_wait_drain(reinterpret_cast<uint64_t*>(s) + 8 + lane, (commits - 1) & 1);
}

// The item that a role works on next (row0 < 0: none is left).  Every thread of the role calls it.
struct Att16Items {
  Att16Bars* s;
  int n = 0;
  __device__ __forceinline__ bool next(Att16Item& it) {
    const int b = n & 1;
    const bool ok = att_wait(&s->ifull[b], (n >> 1) & 1, s);
    it = s->item[b];
    mbar_arrive(&s->iempty[b]);
    ++n;
    return ok && it.row0 >= 0;
  }
};
// Tiles of an item, and those that its second block of rows (y 1) or its first (y 0) sees any key of.
template <int NQ>
struct Att16Tiles {
  int n, a1, b0;  // tiles; block 0: 0 .. a1 - 1, block 1: b0 .. n - 1 (b0 = n: it has no rows)
  __device__ __forceinline__ Att16Tiles(const Att16Item& it, int tb, int window, bool causal) {
    n = (it.hi - it.lo + kAttN - 1) / kAttN;
    a1 = n;
    b0 = n;
    if (NQ == 2 && it.t0 + tb < it.len) {
      b0 = 0;
      if (causal) {
        a1 = (it.t0 + tb - it.lo + kAttN - 1) / kAttN;
        if (window > 0) b0 = max(0, it.t0 + tb - window + 1 - it.lo) / kAttN;
      }
    }
  }
  __device__ __forceinline__ bool sees(int y, int j) const { return y ? j >= b0 : j < a1; }
};

// The slot that the shared pages' names are read from: the first of the batch that holds their `keys` rows (-1: none does).
// A warp's threads call it together.
__device__ __forceinline__ int att_shared_slot(const int* slots, const int* lens, int n_seq, int n_slots, int keys) {
  const int lane = threadIdx.x & 31;
  for (int i0 = 0; i0 < n_seq; i0 += 32) {
    const int slot = i0 + lane < n_seq ? __ldcg(slots + i0 + lane) : -1;
    const unsigned who = __ballot_sync(0xFFFFFFFFu, slot >= 0 && slot < n_slots && __ldcg(lens + max(slot, 0)) >= keys);
    if (who) return __shfl_sync(0xFFFFFFFFu, slot, __ffs(who) - 1);
  }
  return -1;
}

// Finite values hidden from a row do not reach it: their weights are zero.  Hidden infinities and NaNs would, as
// NaN (0 * inf).  So where a row's weights add up to a finite sum and its output holds a NaN, the values that it sees
// are looked at, and if they do not account for it, the row is taken anew, with weights in fp32.
// A warp does this for its rows together (`on`: the lane's row is one of them).  L lanes share a key: each has eight
// columns of the item's values, and of the head dim in one piece or two.  First the keys that all of the rows see are
// searched for values that are not finite, then the few that only some see; rows that are still not accounted for are
// made four at a time, in one pass with a running maximum.  Rare, and bound by the latency of each step's loads and sums: a prompt
// of 4,000 tokens of 512 (8 heads on 1) with a row of NaNs 60 tokens from its end takes 13 ms, one of 16,384 tokens 57 (fp16 75).
// The other roles wait longer than usual meanwhile: `beat` counts the steps (att_wait).
template <int D, bool BF>
__device__ __noinline__ void att_repair(const Att16Args& a, int* beat, bool on, const uint16_t* q, uint16_t* out, int row0, int head,
                                        int half, int first, int last) {
  constexpr int DV = Att16<D>::DV, L = DV / 8, KP = 32 / L, CK = D / DV, R = 4, U = 4, US = 8;
  constexpr uint32_t kAll = 0xFFFFFFFFu, kExp = BF ? 0x7F80u : 0x7C00u;
  const int lane = threadIdx.x & 31, sub = lane / L, col = lane % L * 8;
  const uint16_t* k = a.k + (long)row0 * a.k_row + (long)head * a.k_head + col;
  const uint16_t* v = a.v + (long)row0 * a.v_row + (long)head * a.v_head + half * DV + col;
  auto row_out = [&](int r) {
    return reinterpret_cast<uint16_t*>(__shfl_sync(kAll, reinterpret_cast<unsigned long long>(out), r)) + half * DV + col;
  };
  auto nans = [&](const uint16_t* o) {  // which of the lane's columns hold a NaN
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m |= (uint32_t)((__ldcg(o + e) & 0x7FFFu) > kExp) << e;
    return m;
  };
  auto odd = [&](const uint4& x) {  // which of eight numbers are not finite
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) m |= (uint32_t)((w[e] & kExp) == kExp) << (2 * e) | (uint32_t)((w[e] >> 16 & kExp) == kExp) << (2 * e + 1);
    return m;
  };
  // Those of the columns `want` in which a value of the keys from .. to is not finite; the search ends when all are found.
  auto search = [&](int from, int to, uint32_t want) {
    uint32_t found = 0;
    for (int j0 = from; j0 <= to; j0 += KP * US) {
      uint4 x[US];
#pragma unroll
      for (int u = 0; u < US; ++u) {
        const int j = j0 + u * KP + sub;
        x[u] = j <= to ? *reinterpret_cast<const uint4*>(v + (long)j * a.v_row) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < US; ++u) found |= odd(x[u]);
#pragma unroll
      for (int o = L; o < 32; o <<= 1) found |= __shfl_xor_sync(kAll, found, o);
      if (lane == 0) atomicAdd(beat, 1);
      if (!__any_sync(kAll, want & ~found)) break;
    }
    return found & want;
  };
  uint32_t any = 0;
  unsigned rows = 0;
  for (unsigned m = __ballot_sync(kAll, on); m; m &= m - 1) {
    const int r = __ffs(m) - 1;
    const uint32_t bad = nans(row_out(r));
    if (__any_sync(kAll, bad)) rows |= 1u << r;
    any |= bad;
  }
  if (!rows) return;
  on = rows >> lane & 1;
  const int lo = __reduce_max_sync(kAll, on ? first : 0), hi = __reduce_min_sync(kAll, on ? last : 0x7FFFFFFF);
  const uint32_t seen = search(lo, hi, any);
  unsigned left = 0;
  for (unsigned m = rows; m; m &= m - 1) {
    const int r = __ffs(m) - 1, f = __shfl_sync(kAll, first, r), e = __shfl_sync(kAll, last, r);
    uint32_t bad = nans(row_out(r)) & ~seen;
    if (__any_sync(kAll, bad)) bad &= ~search(f, min(lo - 1, e), bad);
    if (__any_sync(kAll, bad)) bad &= ~search(max(hi + 1, f), e, bad);
    if (__any_sync(kAll, bad)) left |= 1u << r;
  }
  while (left) {
    const uint16_t* qr[R];
    uint16_t* o[R];
    int f[R], e[R], n = 0, j_lo = 0x7FFFFFFF, j_hi = -1, r = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {  // (fewer than R are left: the last one again)
      if (left) {
        r = __ffs(left) - 1;
        left &= left - 1;
        n = i + 1;
      }
      qr[i] = reinterpret_cast<const uint16_t*>(__shfl_sync(kAll, reinterpret_cast<unsigned long long>(q), r)) + col;
      o[i] = row_out(r);
      f[i] = __shfl_sync(kAll, first, r);
      e[i] = __shfl_sync(kAll, last, r);
      j_lo = min(j_lo, f[i]);
      j_hi = max(j_hi, e[i]);
    }
    uint4 qv[R][CK];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int c = 0; c < CK; ++c) qv[i][c] = *reinterpret_cast<const uint4*>(qr[i] + c * DV);
    float acc[R][8], top[R], sum[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      top[i] = -INFINITY;
      sum[i] = 0.f;
#pragma unroll
      for (int x = 0; x < 8; ++x) acc[i][x] = 0.f;
    }
    for (int j0 = j_lo; j0 <= j_hi; j0 += KP * U) {
      uint4 kx[U][CK], vx[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long j = min(j0 + u * KP + sub, j_hi);
#pragma unroll
        for (int c = 0; c < CK; ++c) kx[u][c] = *reinterpret_cast<const uint4*>(k + j * a.k_row + c * DV);
        vx[u] = *reinterpret_cast<const uint4*>(v + j * a.v_row);
      }
      float s[R][U];
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int u = 0; u < U; ++u) s[i][u] = 0.f;
#pragma unroll
      for (int c = 0; c < CK; ++c)
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          float kf[U];
#pragma unroll
          for (int u = 0; u < U; ++u) kf[u] = att_one<BF>(kx[u][c], x);
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const float qf = att_one<BF>(qv[i][c], x);
#pragma unroll
            for (int u = 0; u < U; ++u) s[i][u] = fmaf(qf, kf[u], s[i][u]);
          }
        }
#pragma unroll
      for (int w = 1; w < L; w <<= 1)
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int u = 0; u < U; ++u) s[i][u] += __shfl_xor_sync(kAll, s[i][u], w);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float most = top[i];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + u * KP + sub;
          s[i][u] = j >= f[i] && j <= e[i] ? s[i][u] * a.scale : -INFINITY;
          most = fmaxf(most, s[i][u]);
        }
        const float ref = most == -INFINITY ? 0.f : most, back = att_exp2(top[i] - ref);
        top[i] = most;
        sum[i] *= back;
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[i][x] *= back;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + u * KP + sub;
          const bool sees = j >= f[i] && j <= e[i];
          const float p = att_exp2(s[i][u] - ref);
          sum[i] += p;
#pragma unroll
          for (int x = 0; x < 8; ++x) acc[i][x] = sees ? fmaf(p, att_one<BF>(vx[u], x), acc[i][x]) : acc[i][x];
        }
      }
      if (lane == 0) atomicAdd(beat, 1);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int w = L; w < 32; w <<= 1) {  // the lanes' keys together
        const float most = fmaxf(top[i], __shfl_xor_sync(kAll, top[i], w)), mine = most == -INFINITY ? 0.f : att_exp2(top[i] - most);
        top[i] = most;
        sum[i] *= mine;
        sum[i] += __shfl_xor_sync(kAll, sum[i], w);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          acc[i][x] *= mine;
          acc[i][x] += __shfl_xor_sync(kAll, acc[i][x], w);
        }
      }
      const uint32_t bad = i < n && sub == 0 ? nans(o[i]) : 0u;
      const float inv = sum[i] != 0.f ? 1.f / sum[i] : 0.f;
#pragma unroll
      for (int x = 0; x < 8; ++x)
        if (bad >> x & 1) o[i][x] = (uint16_t)att_pack<BF>(acc[i][x] * inv, 0.f);
      __syncwarp();
    }
  }
}

// The 12 warps begin with 168 registers a thread; softmax warps need 200 or so: 4 x 72 + 8 x 216 = 12 x 168.
__device__ __forceinline__ void att_fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n"); }
__device__ __forceinline__ void att_more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 216;\n"); }

template <int D, bool BF, bool PREFIX>
__global__ void __launch_bounds__(Att16<D>::kThreads, 1)
    att16_kernel(const __grid_constant__ Att16Args a, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap) {
  using C = Att16<D>;
  constexpr int NQ = C::NQ, DV = C::DV;
  extern __shared__ __align__(16) uint8_t att_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(att_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qop = base;
  uint8_t* ring = base + C::kQ;
  Att16Bars* s = reinterpret_cast<Att16Bars*>(ring + C::kStages * C::kStage);
  float* sums = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(s) + 512);  // NQ 1: of an item's rows
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&s->full[i], 1);
      mbar_init(&s->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s->sfull[i], 1);
      mbar_init(&s->pfull[i], 4);
      mbar_init(&s->pvdone[i], 1);
      mbar_init(&s->ifull[i], 1);
      mbar_init(&s->iempty[i], C::kThreads - 32);  // all but the warp that makes them
    }
    mbar_init(&s->qfull, 1);
    mbar_init(&s->qdone, 1);
    mbar_init(&s->vneed, 1);
    mbar_init(&s->vtail, 64);
    mbar_init(&s->lfull, 4);
    mbar_init(&s->odone, 1);
    mbar_init(&s->ofree, 4);
    mbar_init(&s->drained, 1);
    s->abort = 0;
    s->beat = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == C::kSoftWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(su32(&s->tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  tc_fence_before();
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s->tmem;

  // The calling thread's output row of block y of an item, whose weights add up to l, from tensor memory.
  auto give_out = [&](const Att16Item& it, int y, float l) {
    const int row = (warp & 3) * 32 + lane, tok_in = row / a.group, hq = row % a.group, tok = it.t0 + y * a.tb + tok_in;
    const bool on = tok_in < a.tb && tok < it.len;
    const uint32_t from = tmem + ((uint32_t)((warp & 3) * 32) << 16) + y * DV;
    const float factor = PREFIX ? 1.f : l != 0.f ? 1.f / l : 0.f;
    const uint64_t inv = att_two(factor, factor);
    float* part = PREFIX ? a.part_o + ((long)it.part * (NQ * kAttM) + y * kAttM + row) * D + it.half * DV : nullptr;
    uint16_t* out = PREFIX || !on ? nullptr : a.out + (long)(it.row0 + tok) * a.o_row + (long)(it.head * a.group + hq) * a.o_head;
    uint64_t odd = 0ull;  // becomes NaN with a number that is not finite
    uint32_t u[2][32];    // the next 32 numbers come while these are on their way out
    tc_tld32(from, u[0]);
#pragma unroll
    for (int c = 0; c < DV; c += 32) {
      uint32_t(&f)[32] = u[(c >> 5) & 1];
      tc_tld_wait();
      if (c + 32 < DV) tc_tld32(from + c + 32, u[((c >> 5) + 1) & 1]);
      if (NQ == 1 && c + 32 >= DV) {  // all is in registers
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s->ofree);
      }
      if (PREFIX) {
        if (on) {
#pragma unroll
          for (int k = 0; k < 4; ++k) att_store32(part + c + 8 * k, f + 8 * k);
        }
      } else {
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const uint64_t x = att_mul2(att_two(__uint_as_float(f[2 * k]), __uint_as_float(f[2 * k + 1])), inv);
          float f0, f1;
          att_split(x, f0, f1);
          odd = att_fma2(x, 0ull, odd);
          w[k] = att_pack<BF>(f0, f1);
        }
        uint16_t* o = out + it.half * DV + c;
        if (!on) {
        } else if (a.o_vec == 2) {
          att_store32(o, w);
          att_store32(o + 16, w + 8);
        } else if (a.o_vec) {
#pragma unroll
          for (int k = 0; k < 4; ++k) reinterpret_cast<uint4*>(o)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            o[2 * k] = (uint16_t)w[k];
            o[2 * k + 1] = (uint16_t)(w[k] >> 16);
          }
        }
      }
      __syncwarp();
    }
    float odd0, odd1;
    att_split(odd, odd0, odd1);
    const bool spoilt = !PREFIX && on && !(odd0 + odd1 == 0.f) && att_finite(l) && !*reinterpret_cast<volatile int*>(&s->abort);
    __syncwarp();
    if (!PREFIX && __any_sync(0xFFFFFFFFu, spoilt))
      att_repair<D, BF>(a, &s->beat, spoilt, a.q + (long)(it.row0 + tok) * a.q_row + (long)(it.head * a.group + hq) * a.q_head, out, it.row0,
                        it.head, it.half, a.window > 0 ? max(0, tok - a.window + 1) : 0, tok);
    __syncwarp();
  };
  if (warp == C::kSoftWarps + 1) {
    // ------------------------------------------------ items, and their tiles by TMA
    att_fewer_registers();
    const uint32_t one = att_elect();
    int st = 0, lap = 0, copied = 0;  // the ring's stage and lap; items whose queries were asked for
    const int total = PREFIX ? C::HV * a.kvh * a.splits * ((a.n_seq + NQ * a.tb - 1) / (NQ * a.tb)) : 0;
    const int from_slot = PREFIX ? max(0, att_shared_slot(a.slots, a.lens, a.n_seq, a.n_slots, a.keys)) : 0;
    // prompt: the lane's sequence of the 32 from `seq` on: its first row, length and last item (one too far);
    // items of all 32, and of the sequences ahead of them
    int seq = -32, from = 0, len = 0, upto = 0, all = 0, before = 0;
    int lowest = a.n_rows, highest = 0;  // of the rows of the lane's sequences
    int index = blockIdx.x;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      Att16Item it;
      it.row0 = -1;
      if (PREFIX) {
        if (index < total) {
          int x = index;
          it.part = x / C::HV;
          it.half = x % C::HV;
          x /= C::HV;
          const int split = x % a.splits;
          x /= a.splits;
          it.head = x % a.kvh;
          it.t0 = x / a.kvh * (NQ * a.tb);
          it.row0 = 0;
          it.len = a.n_seq;
          it.lo = split * a.tiles_per * kAttN;
          it.hi = min(a.keys, it.lo + a.tiles_per * kAttN);
        }
        index += gridDim.x;
      } else {
        const int blk = index / (a.kvh * C::HV), x = index % (a.kvh * C::HV);
        it.head = x / C::HV;
        it.half = x % C::HV;
        while (blk >= before + all && seq + 32 < a.n_seq) {
          before += all;
          seq += 32;
          const int i = seq + lane;
          from = len = upto = 0;
          if (i < a.n_seq) {
            from = __ldcg(a.offsets + i);
            const int to = __ldcg(a.offsets + i + 1);
            if (from < 0 || to < from || to > a.n_rows) {
              if (blockIdx.x == 0) set_err(a.err, G4_DEV_BAD_POSITION);
            } else {
              len = to - from;
              if (len > 0) {
                lowest = min(lowest, from);
                highest = max(highest, to);
              }
              upto = (len + NQ * a.tb - 1) / (NQ * a.tb);
            }
          }
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += y;
          }
          all = __shfl_sync(0xFFFFFFFFu, upto, 31);
        }
        if (blk < before + all) {
          const int w = __ffs(__ballot_sync(0xFFFFFFFFu, blk < before + upto)) - 1;
          it.row0 = __shfl_sync(0xFFFFFFFFu, from, w);
          it.len = __shfl_sync(0xFFFFFFFFu, len, w);
          // the last tokens, with the most keys, come first
          it.t0 = (__shfl_sync(0xFFFFFFFFu, upto, w) - 1 - (blk - before)) * (NQ * a.tb);
          it.lo = a.window > 0 ? max(0, it.t0 - a.window + 1) : 0;
          it.hi = min(it.t0 + NQ * a.tb, it.len);
        } else {  // all sequences have been looked at: the rows that they span
          it.lo = __reduce_min_sync(0xFFFFFFFFu, lowest);
          it.hi = __reduce_max_sync(0xFFFFFFFFu, highest);
        }
      }
      if (n >= 2) ok = att_wait(&s->iempty[n & 1], ((n - 2) >> 1) & 1, s);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (lane == 0) {
        if (!ok) it.row0 = -1;
        s->item[n & 1] = it;
        mbar_arrive(&s->ifull[n & 1]);
      }
      __syncwarp();
      if (!ok || it.row0 < 0) break;
      const int tiles = (it.hi - it.lo + kAttN - 1) / kAttN;
      int next = 0;
      // NQ 2: keys 0, the queries, values 0, keys 1 ...; NQ 1, whose scores run a tile ahead: the queries, keys 0, keys 1, values 0, ...
      for (int x = 0; x < 2 * tiles && ok; ++x) {
        if (x == (NQ == 2 ? 1 : 0)) {  // (NQ 1: a tile of keys may have to wait for products of this very item)
          if (n) ok = att_wait(&s->qdone, (n - 1) & 1, s);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          const int blocks = NQ == 2 && it.t0 + a.tb < it.len ? 2 : 1, bytes = a.tb * a.group * 128;
          if (lane == 0) mbar_expect_tx(&s->qfull, blocks * (D / 64) * bytes);
          __syncwarp();
          if (lane < blocks * (D / 64)) {
            const int y = lane / (D / 64), z = lane % (D / 64);
            att_tma3(qop + y * (kAttM * D * 2) + z * (kAttM * 128), &qmap, 64 * z, it.head * a.group, it.row0 + it.t0 + y * a.tb, &s->qfull);
          }
          ++copied;
          __syncwarp();
        }
        // the next item, so that its number is there when this one's tiles are on their way (asked for earlier, the last
        // items end unevenly)
        if (!PREFIX && x == 2 * tiles - 2 && lane == 0) next = gridDim.x + atomicAdd(a.ticket, 1u);
        int j;
        bool values;
        if (NQ == 2) {
          j = x >> 1;
          values = x & 1;
        } else {
          values = x == 2 * tiles - 1 || (x >= 2 && !(x & 1));
          j = values ? (x == 2 * tiles - 1 ? tiles - 1 : x / 2 - 1) : (x + 1) / 2;
        }
        const int key = it.lo + j * kAttN;
        const int parts = values ? C::VS : C::KS;
        for (int y = 0; y < parts && ok; ++y) {
          if (lap) ok = att_wait(&s->empty[st], (lap - 1) & 1, s);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          uint8_t* to = ring + st * C::kStage;
          const int rows = values ? C::kVRows : kAttN, from = key + (values ? y * C::kVRows : 0);
          [[maybe_unused]] const int slabs = C::kStage / (rows * 128);
          const int col = values ? it.half * DV : y * slabs * 64;
          const CUtensorMap* map = values ? &vmap : &kmap;
          if (!PREFIX) {
            att_tma4(one, to, map, 0, it.head, it.row0 + from, col / 64, &s->full[st], C::kStage);
          } else {
            // boxes of up to a page; a page that is missing (the join's business) reads page 0
            const int box = min(rows, 1 << a.log_page), boxes = rows / box;
            const int live = min(boxes, max(0, (a.keys - from + box - 1) / box));
            if (lane == 0) mbar_expect_tx(&s->full[st], live * slabs * box * 128);
            __syncwarp();
            if (lane < live * slabs) {
              const int z = lane / live, b = lane % live, at = from + b * box;
              int page = __ldcg(a.table + (long)from_slot * a.max_pages + (at >> a.log_page));
              if (page < 0 || page >= a.n_pages) page = 0;
              att_tma2(to + z * rows * 128 + b * box * 128, map, col + 64 * z,
                       ((page * a.kvh + it.head) << a.log_page) + (at & ((1 << a.log_page) - 1)), &s->full[st]);
            }
            __syncwarp();
          }
          if (++st == C::kStages) st = 0, ++lap;
        }
      }
      if (!PREFIX) index = __shfl_sync(0xFFFFFFFFu, next, 0);
    }
    // every copy that was asked for arrives before the CTA ends
    if (copied) mbar_wait_drain(&s->qfull, (copied - 1) & 1);
    const int asked = lap * C::kStages + st;
    for (int k = max(0, asked - C::kStages); k < asked; ++k) mbar_wait_drain(&s->full[k % C::kStages], (k / C::kStages) & 1);
    __syncwarp();
  } else if (warp == C::kSoftWarps) {
    // ------------------------------------------------ matrix instructions
    att_fewer_registers();
    {
      const uint32_t one = att_elect();
      Att16Items items{s};
      Att16Item it;
      int st = 0, lap = 0, n_p[2] = {0, 0}, tiles_done = 0, tails = 0, second = 0;
      bool ok = true;
      auto stage = [&]() {  // the next stage, filled
        ok = att_wait(&s->full[st], lap & 1, s) && ok;
        tc_fence_after();
        return su32(ring + st * C::kStage);
      };
      auto done = [&]() {
        att_commit(one, &s->empty[st]);
        if (++st == C::kStages) st = 0, ++lap;
      };
      auto scores_part = [&](int y, int buf, uint32_t kaddr, int part) {
        if (!ok) return;
        const uint64_t qd = tc_desc(su32(qop) + y * (kAttM * D * 2) + part * (C::kStage / C::kSlab) * (kAttM * 128), 0), kd = tc_desc(kaddr, 0);
        const uint32_t to = tmem + C::kColS + buf * kAttN;
#pragma unroll
        for (int k = 0; k < C::kStage / C::kSlab * 4; ++k) {
          const uint32_t off = (k >> 2) * C::kSlab + (k & 3) * 32;
          att_mma_ss(one, to, att_desc_at(qd, off), att_desc_at(kd, off), att_idesc<BF>(kAttN, false), part > 0 || k > 0);
        }
      };
      auto weights_part = [&](int y, int buf, uint32_t vaddr, int part, bool first) {
        if (!ok) return;
        const uint64_t vd = tc_desc(vaddr, C::kVRows * 128);
        const uint32_t to = tmem + y * DV, from = tmem + C::kColS + buf * kAttN + part * (C::kVRows / 16) * 8;
#pragma unroll
        for (int k = 0; k < C::kVRows / 16; ++k)
          att_mma_ts(one, to, from + k * 8, att_desc_at(vd, k * 2048), att_idesc<BF>(DV, true), !first || part > 0 || k > 0);
      };
      auto clear_tail = [&]() {  // has the rows of values behind the item's last key cleared, once they are there
        for (int y = 0; y < C::VS; ++y) {
          const int x = st + y < C::kStages ? st + y : st + y - C::kStages;
          ok = att_wait(&s->full[x], (st + y < C::kStages ? lap : lap + 1) & 1, s) && ok;
        }
        if (one) mbar_arrive(&s->vneed);
        ok = att_wait(&s->vtail, tails & 1, s) && ok;
        ++tails;
        tc_fence_after();
      };
      while (items.next(it)) {
        const Att16Tiles<NQ> t(it, a.tb, a.window, !PREFIX);
        const bool tail = att_past_end<PREFIX>(it);
        ok = att_wait(&s->qfull, (items.n - 1) & 1, s) && ok;
        tc_fence_after();
        if (NQ == 2) {
          second += t.b0 < t.n;
          uint32_t k0 = stage();
          for (int y = 0; y < 2; ++y)
            if (t.sees(y, 0)) {
              scores_part(y, y, k0, 0);
              att_commit(one, &s->sfull[y]);
            }
          done();
          if (t.n == 1) att_commit(one, &s->qdone);
          for (int j = 0; j < t.n; ++j) {
            const uint32_t v0 = stage();
            if (tail && j == t.n - 1) clear_tail();
            const int vst = st, vlap = lap;
            uint32_t k1 = 0;
            bool have = false;
            for (int y = 0; y < 2; ++y) {
              if (t.sees(y, j)) {
                ok = att_wait(&s->pfull[y], n_p[y] & 1, s) && ok;
                ++n_p[y];
                tc_fence_after();
                weights_part(y, y, v0, 0, y ? j == t.b0 : j == 0);
                if (!t.sees(y, j + 1) || j + 1 == t.n) att_commit(one, &s->pvdone[y]);  // (else the next scores tell it)
              }
              if (y == 1) att_commit(one, &s->empty[vst]);
              if (j + 1 < t.n && t.sees(y, j + 1)) {
                if (!have) {
                  const int kst = vst + 1 == C::kStages ? 0 : vst + 1, klap = vst + 1 == C::kStages ? vlap + 1 : vlap;
                  ok = att_wait(&s->full[kst], klap & 1, s) && ok;
                  tc_fence_after();
                  k1 = su32(ring + kst * C::kStage);
                  have = true;
                }
                scores_part(y, y, k1, 0);
                att_commit(one, &s->sfull[y]);
              }
            }
            if (++st == C::kStages) st = 0, ++lap;
            if (j + 1 < t.n) {
              done();
              if (j + 2 == t.n) att_commit(one, &s->qdone);
            }
          }
        } else {
          auto scores = [&](int j) {
            const int b = (tiles_done + j) & 1;
            for (int y = 0; y < C::KS; ++y) {
              scores_part(0, b, stage(), y);
              done();
            }
            att_commit(one, &s->sfull[b]);
            if (j == t.n - 1) att_commit(one, &s->qdone);
          };
          scores(0);
          for (int j = 0; j < t.n; ++j) {
            const int b = (tiles_done + j) & 1;
            if (j + 1 < t.n) scores(j + 1);
            for (int y = 0; y < C::VS; ++y) {
              const uint32_t v0 = stage();
              if (y == 0) {
                if (tail && j == t.n - 1) clear_tail();
                if (j == 0 && items.n > 1) ok = att_wait(&s->ofree, items.n & 1, s) && ok;  // the item before has been read
                ok = att_wait(&s->pfull[b], n_p[b] & 1, s) && ok;
                ++n_p[b];
                tc_fence_after();
              }
              weights_part(0, b, v0, y, j == 0);
              done();
            }
            att_commit(one, &s->pvdone[0]);
          }
          att_commit(one, &s->odone);
          tiles_done += t.n;
        }
      }
      att_commit(one, &s->drained);
      mbar_wait_drain(&s->drained, 0);
      const int whole = items.n - 1;
      att_last(s, C::kStages, st, lap, n_p[0], n_p[1], NQ == 2 ? whole : tiles_done, second, whole, NQ == 1 ? whole : 0);
    }
    __syncwarp();
  } else if (warp == C::kSoftWarps + 2 || warp == C::kSoftWarps + 3) {
    // ------------------------------------------------ values behind the last key; rows of no sequence
    att_fewer_registers();
    const int me = threadIdx.x - 32 * (C::kSoftWarps + 2);
    constexpr int CH = D / 8;  // 16-byte pieces of a row
    Att16Items items{s};
    Att16Item it;
    int st = 0, tails = 0;  // stages and cleared tiles of the items so far
    while (items.next(it)) {
      const int tiles = (it.hi - it.lo + kAttN - 1) / kAttN, live = it.hi - it.lo - (tiles - 1) * kAttN;
      st += tiles * (C::KS + C::VS);
      if (att_past_end<PREFIX>(it)) {  // from the item's last key on: no row of it sees more
        att_wait(&s->vneed, tails++ & 1, s);
        for (int y = 0; y < C::VS; ++y) {
          const int x = st - C::VS + y;
          uint8_t* v = ring + (x % C::kStages) * C::kStage;
          const int first = min(max(live - y * C::kVRows, 0), C::kVRows), pieces = (C::kVRows - first) * 8;
          for (int z = 0; z < DV / 64; ++z)
            for (int e = me; e < pieces; e += 64)
              *reinterpret_cast<uint4*>(v + z * (C::kVRows * 128) + first * 128 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        mbar_arrive(&s->vtail);
      }
    }
    if (!PREFIX && a.zero_rest && !*reinterpret_cast<volatile int*>(&s->abort)) {
      // in front of and behind every sequence: where offsets fall, the first and the last need not be the outermost
      int front = min(max(__ldcg(a.offsets), 0), a.n_rows), end = min(max(__ldcg(a.offsets + a.n_seq), front), a.n_rows);
      front = min(front, it.lo);
      end = max(end, it.hi);
      const int rest = front + a.n_rows - end, heads = a.kvh * a.group;
      for (long e = blockIdx.x * 64 + me; e < (long)rest * heads * CH; e += gridDim.x * 64) {
        const int c = (int)(e % CH), x = (int)(e / CH % heads), r = (int)(e / CH / heads);
        uint16_t* o = a.out + (long)(r < front ? r : end + r - front) * a.o_row + (long)x * a.o_head + 8 * c;
        if (a.o_vec) {
          *reinterpret_cast<uint4*>(o) = make_uint4(0u, 0u, 0u, 0u);
        } else {
          for (int y = 0; y < 8; ++y) o[y] = 0;
        }
      }
    }
  } else if (NQ == 1 && warp >= C::kSoftWarps + 4) {
    // ------------------------------------------------ outputs, while the next item's scores and weights are made
    Att16Items items{s};
    Att16Item it;
    while (items.next(it)) {
      att_wait(&s->lfull, (items.n - 1) & 1, s);
      const float l = sums[(warp & 3) * 32 + lane];
      att_wait(&s->odone, (items.n - 1) & 1, s);
      __syncwarp();
      tc_fence_after();
      give_out(it, 0, l);
    }
  } else {
    // ------------------------------------------------ softmax: a query row per thread
    att_more_registers();
    const int y = warp >> 2, row_in = threadIdx.x & 127, tok_in = row_in / a.group;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ocol = lane_base + y * DV;
    Att16Items items{s};
    Att16Item it;
    int n = 0, done = 0;  // tiles of this block of rows and items so far
    while (items.next(it)) {
      const Att16Tiles<NQ> t(it, a.tb, a.window, !PREFIX);
      const int block0 = it.t0 + y * a.tb;  // the block's first token
      const bool on = tok_in < a.tb && block0 + tok_in < it.len;
      const int j0 = y ? t.b0 : 0, j1 = y ? t.n : t.a1;
      if (j0 >= j1) continue;
      const int tok = min(block0 + min(tok_in, a.tb - 1), it.len - 1);
      // keys that the row sees: first .. last; every row of the block sees all_first .. all_last
      int first = it.lo, last = it.hi - 1, all_first = it.lo, all_last = it.hi - 1;
      if (!PREFIX) {
        last = tok;
        all_last = block0;
        if (a.window > 0) {
          first = max(0, tok - a.window + 1);
          all_first = max(0, min(block0 + a.tb, it.len) - a.window);
        }
      }
      const int warp_last = __reduce_max_sync(0xFFFFFFFFu, last), warp_first = __reduce_min_sync(0xFFFFFFFFu, first);
      float m = -INFINITY, ref = 0.f, l = 0.f;
      // The reference for a largest score mx of tile j; the sum and the output so far follow.
      auto refer = [&](float mx, int j) {
        const bool raise = mx > m + 8.f || (m == -INFINITY && mx > m);
        if (!__any_sync(0xFFFFFFFFu, raise)) return;
        const float nm = raise ? mx : m, fac = raise ? att_exp2(m - nm) : 1.f;
        m = nm;
        ref = m == -INFINITY ? 0.f : m - att_up<BF>();
        l *= fac;
        if (j == j0) return;
        if (NQ == 1) {  // when the previous tile's product is in (NQ 2: it came before the scores); it is the newest that can be
          att_wait(&s->pvdone[0], (n - 1) & 1, s);
          __syncwarp();
          tc_fence_after();
        }
#pragma unroll 1
        for (int c = 0; c < DV; c += 32) {
          uint32_t u[32];
          tc_tld32(ocol + c, u);
          tc_tld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * fac);
          tc_tst32(ocol + c, u);
        }
        tc_tst_wait();
      };
      // A tile of which every row of the block sees every key: the scores stay in registers.
      auto whole_tile = [&](int j, uint32_t cols) {
        uint32_t v[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc_tld32(cols + 32 * c, v + 32 * c);
        tc_tld_wait();
        float top[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) top[k] = fmaxf(__uint_as_float(v[k]), __uint_as_float(v[4 + k]));
#pragma unroll
        for (int k = 8; k < 128; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) top[e] = att_max3(top[e], __uint_as_float(v[k + e]), __uint_as_float(v[k + 4 + e]));
        refer(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale, j);
        const uint64_t sc = att_two(a.scale, a.scale), off = att_two(-ref, -ref);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int k = 0; k < 64; ++k) {
          const uint64_t x = att_fma2(att_two(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), sc, off);
          float p0, p1;
          att_split(x, p0, p1);
          p0 = att_exp2(p0);
          p1 = att_exp2(p1);
          sum[k & 1] = att_add2(sum[k & 1], att_two(p0, p1));
          v[k] = att_pack<BF>(p0, p1);
        }
        tc_tst32(cols, v);
        tc_tst32(cols + 32, v + 32);
        float s0, s1;
        att_split(att_add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      };
      // Any other tile, 32 columns at a time: those of which no row of the warp sees a key are passed over.  (The
      // weights of columns 32 c .. lie where the scores of columns 16 c .. did, which have been read by then.)
      auto edge_tile = [&](int j, int key, uint32_t cols) {
        auto scores = [&](int c, uint32_t (&u)[32]) {
          const int most = last - key - c, least = first - key - c;
          tc_tld32(cols + c, u);
          tc_tld_wait();
          if (key + c + 31 > all_last) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (k > most) u[k] = 0xFF800000u;
          }
          if (key + c < all_first) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (k < least) u[k] = 0xFF800000u;
          }
        };
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < kAttN; c += 32) {
          if (key + c > warp_last || key + c + 31 < warp_first) continue;
          uint32_t u[32];
          scores(c, u);
          float top[2] = {mx, mx};
#pragma unroll
          for (int k = 0; k < 32; k += 4)
#pragma unroll
            for (int e = 0; e < 2; ++e) top[e] = att_max3(top[e], __uint_as_float(u[k + e]), __uint_as_float(u[k + 2 + e]));
          mx = fmaxf(top[0], top[1]);
        }
        refer(mx * a.scale, j);
        const uint64_t sc = att_two(a.scale, a.scale), off = att_two(-ref, -ref);
        uint64_t sum = 0ull;
#pragma unroll 1
        for (int c = 0; c < kAttN; c += 32) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) w[k] = 0u;
          if (key + c <= warp_last && key + c + 31 >= warp_first) {
            uint32_t u[32];
            scores(c, u);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const uint64_t x = att_fma2(att_two(__uint_as_float(u[2 * k]), __uint_as_float(u[2 * k + 1])), sc, off);
              float p0, p1;
              att_split(x, p0, p1);
              p0 = att_exp2(p0);
              p1 = att_exp2(p1);
              sum = att_add2(sum, att_two(p0, p1));
              w[k] = att_pack<BF>(p0, p1);
            }
          }
          tc_tst16(cols + c / 2, w);
        }
        float s0, s1;
        att_split(sum, s0, s1);
        l += s0 + s1;
      };
      for (int j = j0; j < j1; ++j, ++n) {
        const int b = NQ == 2 ? y : n & 1, key = it.lo + j * kAttN;
        const uint32_t cols = lane_base + C::kColS + b * kAttN;
        att_wait(&s->sfull[b], (NQ == 2 ? n : n >> 1) & 1, s);
        __syncwarp();
        tc_fence_after();
        if (key + kAttN - 1 > all_last || key < all_first) edge_tile(j, key, cols);
        else whole_tile(j, cols);
        tc_tst_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          // the previous tile's product, long in by now: no arrival at pvdone goes unseen, so that a phase stands for one tile
          if (NQ == 1 && n > 0) att_wait(&s->pvdone[0], (n - 1) & 1, s);
          mbar_arrive(&s->pfull[b]);
        }
        __syncwarp();
      }
      if (NQ == 2) {
        att_wait(&s->pvdone[y], done++ & 1, s);
        __syncwarp();
        tc_fence_after();
        give_out(it, y, l);
      } else {
        if (items.n > 1) att_wait(&s->ofree, items.n & 1, s);  // the item before has been read, its sums too
        sums[row_in] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s->lfull);
      }
      if (PREFIX && on && it.half == 0) a.part_ml[(long)it.part * (NQ * kAttM) + y * kAttM + row_in] = make_float2(m == -INFINITY ? m : ref, l);
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    if (s->abort) set_err(a.err, G4_DEV_TIMEOUT);
    if (!PREFIX) {  // the last CTA puts the counters back
      __threadfence();
      if (atomicAdd(a.ticket + 1, 1u) == gridDim.x - 1) {
        a.ticket[0] = 0;
        a.ticket[1] = 0;
      }
    }
  }
  if (warp == C::kSoftWarps) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512) : "memory");
  }
}

}  // namespace g4
