// Attention of blocks of query tokens over the 4-bit cache on the 5th-generation tensor cores,
// for bf16 queries with more than kv4_block_rows query rows (tokens x heads) per KV head and head
// dims up to 256; and the account of the weights the rows received.
//
// An item is 128 query rows of one KV head.  Four warps decode tiles of 64 keys, and four of values,
// once for all 128 rows into 128-byte-swizzled shared memory; per pair of tiles
//   S = Q K^T  (both operands shared, 128 x 128, fp32 in tensor memory)
// and per tile
//   P = 2^(scale S - m) on four warps, a row per thread, to tensor memory as bf16 parts
//   O += P V   (A tensor memory, B shared with the head dim leading, 128 x D in tensor memory)
// S is free again as soon as the four warps hold its second half in registers, so the next
// pair's S is made while they take exponentials.  A product whose A operand lies in tensor
// memory takes about 125 cycles per 16 numbers of depth however narrow it is: with Q there and
// 64 keys at a time the scores alone took 2,000 of 3,400 cycles a tile.
// P goes in two parts (p - bf16(p) as well), so 16 bits of every weight count; the second pass
// costs 150 cycles a tile.  A row's reference m is raised, and its sums rescaled, only when a
// score exceeds it by 2^8: weights up to 256 lose nothing in fp32 or in the parts.
// Tensor memory holds O (D columns), S (128) and P (2 x 64): all 512 columns at D = 256.
//
// The account (ACCOUNT): the same pipeline without values: a CTA owns a run of keys, takes every
// block of 128 query rows past them, and adds up p = 2^(scale S - lse) over the rows, by a
// butterfly over the lanes that leaves each lane two columns, in a fixed order.  There the
// queries lie in tensor memory, twice, filled ahead by four warps of their own, S has two
// buffers, and so have the decoded keys.
//
// Eight sequences of up to 8,000 rows, 512 query rows each (64 tokens, eight heads of 256): attention 54
// us (26.1 GFLOP, 0.48 PFLOP/s; 39.1 and 0.72 with the weights' second part), join 13, account 43 (13.0
// GFLOP).  The tensor cores are busy 40% of the first; what bounds it is the chain scores ->
// exponentials -> product of each pair of tiles on 128 softmax threads, with the decoding behind it.
// Compiled, the attention spills 8 to 20 bytes of its 128 registers a thread.
#pragma once
#include "kv4_attend.cuh"

namespace g4 {

// More query rows than this per KV head take these kernels.  Their cost hardly depends on the rows up
// to 128 an item; the other path decodes the keys once per eight rows.  Measured (bf16, eight query
// heads on one KV head; microseconds here / on the other path; with the account, without it):
//                 eight sequences of 8,000 rows      of 2,000                     one of 200
//   D = 64,  96:    50.7 / 47.0,   32.8 / 24.6    36.2 / 36.5,  24.0 / 16.5    20.1 / 24.5
//           128:    53.8 / 55.9,   36.8 / 28.7    37.5 / 41.2,  25.4 / 16.5    20.4 / 28.6
//   D = 128, 64:    52.2 / 54.6,   34.9 / 28.7    36.7 / 32.9,  24.7 / 18.3    22.6 / 22.7
//            80:    52.8 / 61.4,   35.6 / 29.5    37.4 / 36.9,  24.7 / 18.6    23.3 / 25.1
//   D = 256, 48:    63.9 / 67.0,   43.0 / 34.9    41.6 / 38.8,  28.3 / 22.4    26.6 / 24.8
//            64:    64.0 / 79.1,   43.7 / 40.5    41.1 / 43.2,  28.6 / 22.8    26.7 / 28.4
//           512:   108.8 / 444,    63.2 / 209     62.5 / 186,   37.9 / 69.8    34.8 / 113
// The border is where the account's calls break even: those without it would still gain a few
// microseconds beyond, but a call's numbers do not depend on whether it accumulates.
__host__ __device__ constexpr int kv4_block_rows(int d) { return d == 64 ? 96 : d == 128 ? 64 : 48; }
constexpr int kKv4M = 128;          // query rows of an item
constexpr int kKv4N = 64;           // keys of a tile
constexpr int kKv4RunTiles = 16;    // account: tiles of a run at the most (8 and 32 take the same time: their
                                    // gains lie in shared memory, and few CTAs have longer runs)
constexpr int kKv4BlockThreads = 512;

template <int D, bool ACCOUNT>
struct Kv4Blk {
  static constexpr int kHalf = 9 * D;                       // coded keys (or values) of a block
  static constexpr int kTile = 4 * kHalf;                   // and of a tile: a ring stage
  static constexpr int kKRing = ACCOUNT ? 3 : 2, kVRing = ACCOUNT ? 0 : 1;  // stages: what fits beside the operands
  static constexpr int kOperand = kKv4N * D * 2;            // decoded keys or values of a tile
  static_assert(2 * kOperand >= kKv4MaxSlots * 4, "the plan's table of slots lies where the keys will");
  static constexpr int kKBufs = ACCOUNT ? 2 : 1;            // pairs of decoded key tiles
  static constexpr int kSBufs = kKBufs;
  static constexpr int kCols = 512;
  static constexpr int kColQ = 0, kColS = D, kColP = D + 128;  // attention: O at 0; account: Q twice
  static constexpr int kFixed = 512 /* barriers and flags */ + (ACCOUNT ? 4 * kKv4RunTiles * kKv4N * 4 : 0);
  static constexpr int kOps = (ACCOUNT ? 4 : 6) * kOperand; // keys 2 x 2; or queries 2, keys 2, values 2
  static __host__ __device__ size_t smem(int n_seq) {
    return 1024 + (size_t)kOps + (kKRing + kVRing) * kTile + kFixed + (size_t)n_seq * 20 + 16;
  }
};

struct Kv4BlockBars {
  uint64_t full[4], empty[4], kfull[2], kempty[2], vfull[2], sfull[2], sread[2], qfull[2], qdone[2], pfull[2], pvdone[2], drained;
  uint32_t held[2][16];  // blocks of a tile that hold rows, as its keys and values come; a producer is at
                         // most ten tiles ahead of a reader
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Kv4BlockBars) <= 512, "barriers");

__device__ __forceinline__ bool kv4_wait(uint64_t* b, uint32_t parity, Kv4BlockBars* s) {
  if (mbar_try(b, parity)) return true;
  if (*reinterpret_cast<volatile int*>(&s->abort)) return false;
  if (mbar_wait(b, parity, reinterpret_cast<volatile int*>(&s->abort))) return true;
  *reinterpret_cast<volatile int*>(&s->abort) = 1;
  return false;
}
__device__ __forceinline__ void kv4_commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ void kv4_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void kv4_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void kv4_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void kv4_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
// 32 columns of the calling thread's lane, no wait.
__device__ __forceinline__ void kv4_tld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void kv4_tst32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void kv4_tld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void kv4_tst_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Shared-memory operand descriptor, 128-byte swizzle, rows of 128 bytes in groups of eight 1,024
// bytes apart.  Keys: the head dim runs along the rows (`lead` unused).  Values: the head dim is
// the operand's leading dimension and `lead` the distance between its 64-wide slabs.
__device__ __forceinline__ uint64_t kv4_desc(uint32_t saddr, uint32_t lead) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(lead ? lead >> 4 : 1) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// kind::f16: bf16 operands, fp32 result, M 128.
__device__ __forceinline__ constexpr uint32_t kv4_idesc(int n, bool b_leading) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_leading ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kKv4M >> 4) << 24);
}

// ------------------------------------------------------------------------- decoding
// Bank conflicts: eight lanes store 16 bytes at a time, lanes 4 (g & 1) + t of a phase.  A store
// address is row R = g or 2t + .., chunk c of its 128 bytes at c ^ (R & 7).  Keys: the lane's
// chunks are taken in an order permuted by its t and g (and its words swapped into that order by
// selects); values: lanes of odd g store the odd row of a pair first.  Both make the eight
// addresses of a phase distinct modulo 128 bytes.
__device__ __forceinline__ void kv4_cswap(bool swap, uint32_t& a, uint32_t& b) {
  const uint32_t x = swap ? b : a, y = swap ? a : b;
  a = x;
  b = y;
}
// The codes and scales of a block go to registers first, so the ring's stage is free while they
// are decoded.
template <int D>
struct Kv4BlockKeys {
  static constexpr int W = D / 32;
  uint32_t w[2][W];  // rows g and g + 8
  Kv4KeyScales<D> ks[2];
  __device__ __forceinline__ void load(const uint8_t* blk, bool on, int lane) {
    using O = Kv4Off<D>;
    if (!on) {  // zeros
#pragma unroll
      for (int i = 0; i < W; ++i) w[0][i] = w[1][i] = 0u;
      ks[0] = ks[1] = {};
      return;
    }
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(blk)[i * 32 + lane];
      w[0][2 * i] = u.x;
      w[0][2 * i + 1] = u.y;
      w[1][2 * i] = u.z;
      w[1][2 * i + 1] = u.w;
    }
    ks[0] = kv4_key_scales<D>(blk + O::kKs, lane >> 2, lane & 3);
    ks[1] = kv4_key_scales<D>(blk + O::kKs, (lane >> 2) + 8, lane & 3);
  }
  // As block b (0-7) of a pair of tiles into the operand at `to`.
  template <bool WIDE>
  __device__ __forceinline__ void store(int b, uint8_t* to, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int x = D == 256 ? t | (g & 1) << 2 : D == 128 ? t >> 1 | (g & 1) << 1 : 0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int R = 16 * b + 8 * half + g;
      uint32_t(&v)[W] = w[half];
      if constexpr (W >= 4) {
#pragma unroll
        for (int i = 0; i < W; i += 2) kv4_cswap(x & 1, v[i], v[i + 1]);
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (!(i & 2)) kv4_cswap(x & 2, v[i], v[i + 2]);
      }
      uint32_t first = ks[half].two(0), second = D == 256 ? ks[half].two(1) : first;
      if constexpr (W == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) kv4_cswap(x & 4, v[i], v[i + 4]);
        kv4_cswap(x & 4, first, second);
      }
      const Kv4Scale<WIDE> s0(first), s1(second);
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const int n0 = t * (D / 4) + 8 * (j ^ x);  // numbers n0 .. n0 + 7
        const Kv4Scale<WIDE>& s = j < 4 ? s0 : s1;
        *reinterpret_cast<uint4*>(to + (n0 >> 6) * (2 * kKv4N * 128) + R * 128 + ((((n0 >> 3) & 7) ^ (R & 7)) << 4)) =
            make_uint4(s.template pair<0>(v[j]), s.template pair<1>(v[j]), s.template pair<2>(v[j]), s.template pair<3>(v[j]));
      }
    }
  }
};
template <int D>
struct Kv4BlockValues {
  uint4 u[D / 64];  // row pair t: x, y; pair t + 4: z, w
  uint32_t sv[2];
  __device__ __forceinline__ void load(const uint8_t* blk, bool on, int lane) {  // blk: the coded values
    using O = Kv4Off<D>;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) u[i] = on ? reinterpret_cast<const uint4*>(blk)[i * 32 + lane] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int half = 0; half < 2; ++half)
      sv[half] = on ? *reinterpret_cast<const uint32_t*>(blk - O::kV + O::v_scale(2 * t + 8 * half, g * (D / 8) / kKv4Group)) : 0u;
  }
  // As block b (0-3) of a tile into the operand at `to`.
  template <bool WIDE>
  __device__ __forceinline__ void store(int b, uint8_t* to, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int odd = D == 64 ? 0 : g & 1;
    const uint32_t take_a = odd ? 0x7632u : 0x5410u, take_b = odd ? 0x5410u : 0x7632u;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int Ra = 16 * b + 8 * half + 2 * t + odd, Rb = Ra ^ 1;
      const Kv4Scale<WIDE> s(sv[half]);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint32_t p = half ? u[i].z : u[i].x, q = half ? u[i].w : u[i].y;
        const uint32_t y[8] = {s.template pair<0>(p), s.template pair<1>(p), s.template pair<2>(p), s.template pair<3>(p),
                               s.template pair<0>(q), s.template pair<1>(q), s.template pair<2>(q), s.template pair<3>(q)};
        const int n0 = g * (D / 8) + 8 * i;
        uint8_t* slab = to + (n0 >> 6) * (kKv4N * 128);
        const int c = (n0 >> 3) & 7;
        *reinterpret_cast<uint4*>(slab + Ra * 128 + ((c ^ (Ra & 7)) << 4)) =
            make_uint4(__byte_perm(y[0], y[1], take_a), __byte_perm(y[2], y[3], take_a), __byte_perm(y[4], y[5], take_a), __byte_perm(y[6], y[7], take_a));
        *reinterpret_cast<uint4*>(slab + Rb * 128 + ((c ^ (Rb & 7)) << 4)) =
            make_uint4(__byte_perm(y[0], y[1], take_b), __byte_perm(y[2], y[3], take_b), __byte_perm(y[4], y[5], take_b), __byte_perm(y[6], y[7], take_b));
      }
    }
  }
};

// The queries of a row (zeros when it is none) into its lane of tensor memory, bf16 pairs.
template <int D>
__device__ __forceinline__ void kv4_load_queries(const Kv4AttendArgs& a, const Kv4Run& r, int row, uint32_t addr) {
  const bool on = row < r.m * a.group;
  const uint16_t* p = reinterpret_cast<const uint16_t*>(a.q.p);
  if (on) p += (long)r.seq * a.q.seq + (long)(row / a.group) * a.q.row + (long)(r.head * a.group + row % a.group) * a.q.head;
#pragma unroll
  for (int c0 = 0; c0 < D; c0 += 128) {  // up to 256 bytes in flight
    constexpr int N = D < 128 ? 64 : 128;
    uint32_t u[N / 2];
#pragma unroll
    for (int e = 0; e < N / 16; ++e) {
      uint32_t(&w)[8] = *reinterpret_cast<uint32_t(*)[8]>(u + 8 * e);
      const uint16_t* q = p + c0 + 16 * e;
      if (!on) {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = 0u;
      } else if (a.q.vec == 2) {
        kv4_load32b(q, w);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = (uint32_t)__ldcg(q + 2 * k) | ((uint32_t)__ldcg(q + 2 * k + 1) << 16);
      }
    }
#pragma unroll
    for (int c = 0; c < N / 64; ++c) kv4_tst32(addr + c0 / 2 + c * 32, u + 32 * c);
  }
  kv4_tst_wait();
}

// The queries of an item's 128 rows into a swizzled operand, by four warps of 32 rows each: a
// warp copies whole rows, so its loads are contiguous; its lanes work the rows' addresses out
// beforehand, one each.
template <int D>
__device__ __forceinline__ void kv4_share_queries(const Kv4AttendArgs& a, const Kv4Run& r, int row0, uint8_t* to, int tid) {
  constexpr int CH = D / 8, RP = 32 / CH;  // 16-byte chunks of a row, rows a warp copies at a time
  const int lane = tid & 31, mine = row0 + tid, sub = lane / CH, c = lane % CH;
  const uint16_t* p = reinterpret_cast<const uint16_t*>(a.q.p);
  const bool mine_on = mine < r.m * a.group;
  if (mine_on) p += (long)r.seq * a.q.seq + (long)(mine / a.group) * a.q.row + (long)(r.head * a.group + mine % a.group) * a.q.head;
  const unsigned on_mask = __ballot_sync(0xFFFFFFFFu, mine_on);
#pragma unroll 4
  for (int k = 0; k < 32; k += RP) {
    const int from = k + sub, R = (tid & ~31) + from;
    const uint16_t* src = reinterpret_cast<const uint16_t*>(__shfl_sync(0xFFFFFFFFu, (unsigned long long)p, from)) + 8 * c;
    const bool on = (on_mask >> from) & 1;
    uint8_t* dst = to + (c >> 3) * (kKv4M * 128) + R * 128 + (((c & 7) ^ (R & 7)) << 4);
    if (a.q.vec) {
      cp_async16(dst, src, on);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = on ? (uint32_t)__ldcg(src + 2 * e) | ((uint32_t)__ldcg(src + 2 * e + 1) << 16) : 0u;
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  cp_async_wait_all();
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}

// Products of a score and its scale go to exponentials relative to a reference (kv4_exp2), fused with
// the subtraction: rounding the 64 scores of every tile first costs 4 us of the case above.
//
// In the attention all weights of a row share the reference, and what a fused product keeps, up to
// 2^-25 of it, cancels in the division by their sum; it only has to stay in range.  From references
// of 2^31 on the factor becomes the power of two below the scale, whose product with the largest
// score is exact.  Scores that differ at all there differ by 64 or more, so their weights are nothing
// under either factor.
//
// In the account the product's rest would stay in the weight.  Warps with a reference beyond 2^12
// round their products first.
constexpr float kKv4FarAttention = 0x1p31f, kKv4FarAccount = 4096.f;
__device__ __forceinline__ float kv4_power_below(float x) { return __uint_as_float(__float_as_uint(x) & 0x7F800000u); }
__device__ __forceinline__ void kv4_round_far(float (&f)[64], float sc, float fused) {
  if (fused == sc) return;
#pragma unroll
  for (int k = 0; k < 64; ++k) f[k] = __fmul_rn(f[k], sc);
}

// The run of tiles at `at`: for the account, of at most kKv4RunTiles tiles (a.row_tiles 1), with
// `blocks` blocks of 128 query rows to take past them.
template <bool ACCOUNT>
__device__ __forceinline__ Kv4Run kv4_block_run(const Kv4AttendArgs& a, const int* first, const int4* seqs, int at, int g1, int* blocks) {
  const Kv4Run r = kv4_run<kKv4N>(a, first, seqs, at, ACCOUNT ? min(g1, at + kKv4RunTiles) : g1);
  *blocks = ACCOUNT ? (r.m * a.group + kKv4M - 1) / kKv4M : 1;
  return r;
}

template <int D, bool ACCOUNT>
__global__ void __launch_bounds__(kKv4BlockThreads, 1) kv4_block_kernel(const __grid_constant__ Kv4AttendArgs a) {
  using C = Kv4Blk<D, ACCOUNT>;
  using O = Kv4Off<D>;
  extern __shared__ __align__(16) uint8_t kv4_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(kv4_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* kop = base;                                             // [kKBufs] decoded keys of a pair of tiles
  uint8_t* qop = base + 2 * C::kOperand;                           // attention: queries
  uint8_t* vop = base + 4 * C::kOperand;                           // attention: [2] decoded values of a tile
  uint8_t* ring = base + C::kOps;
  Kv4BlockBars* s = reinterpret_cast<Kv4BlockBars*>(ring + (C::kKRing + C::kVRing) * C::kTile);
  float* gacc = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(s) + 512);  // account: [4 warps][keys of a run]
  int4* seqs = reinterpret_cast<int4*>(reinterpret_cast<uint8_t*>(s) + C::kFixed);
  int* first = reinterpret_cast<int*>(seqs + a.n_seq);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kKRing + C::kVRing; ++i) {  // keys' stages, then values'
      mbar_init(&s->full[i], 1);
      mbar_init(&s->empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s->kfull[i], 8);  // two tiles of four warps
      mbar_init(&s->kempty[i], 1);
      mbar_init(&s->vfull[i], 4);
      mbar_init(&s->sfull[i], 1);
      mbar_init(&s->sread[i], 128);
      mbar_init(&s->qfull[i], 128);
      mbar_init(&s->qdone[i], 1);
      mbar_init(&s->pfull[i], 128);
      mbar_init(&s->pvdone[i], 1);
    }
    mbar_init(&s->drained, 1);
    s->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(su32(&s->tmem)), "r"(C::kCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  kv4_fence_before();
  pdl_wait();
  pdl_trigger();
  const int wide = __ldcg(a.c.wide) | a.plain;
  kv4_plan<kKv4N>(a, first, seqs, reinterpret_cast<int*>(kop), !ACCOUNT && blockIdx.x == 0);
  kv4_fence_after();
  const uint32_t tmem = s->tmem;
  const int total = first[a.n_seq], span = kv4_span(a, first, gridDim.x);
  const int g0 = (int)min((unsigned)total, blockIdx.x * (unsigned)span), g1 = (int)min((unsigned)total, (unsigned)g0 + span);

  if (warp == 0 || (!ACCOUNT && warp == 2)) {
    // ------------------------------------------------ producers: coded keys (warp 0), values (warp 2)
    const int part = warp >> 1, ring0 = part * C::kKRing, stages = part ? 1 : C::kKRing;
    int n = 0;
    bool stop = false;
    for (int at = g0; at < g1 && !stop;) {
      int blocks;
      const Kv4Run r = kv4_block_run<ACCOUNT>(a, first, seqs, at, g1, &blocks);
      const int lo = a.window > 0 ? max(0, r.len - r.m + 1 - a.window) : 0;
      for (int x = 0; x < blocks * r.tiles; ++x, ++n) {
        const int b = (r.tile + x % r.tiles) * 4 + lane, st = ring0 + n % stages;
        const bool want = lane < 4 && b * kKv4Block < r.len && b * kKv4Block + kKv4Block > lo;
        const long at_b = want ? kv4_block(a.c, r.slot, r.head, b) : -2;
        if (at_b == -1) set_err(a.c.err, G4_DEV_BAD_POSITION);
        const uint32_t have = __ballot_sync(0xFFFFFFFFu, at_b >= 0);
        if (n >= stages) kv4_wait(&s->empty[st], (n / stages - 1) & 1, s);
        stop = __any_sync(0xFFFFFFFFu, *reinterpret_cast<volatile int*>(&s->abort));
        if (stop) break;
        if (lane == 0) {
          s->held[part][n & 15] = have;
          mbar_expect_tx(&s->full[st], __popc(have) * C::kHalf);
        }
        __syncwarp();
        if (at_b >= 0)
          bulk_g2s(ring + (size_t)st * C::kTile + lane * C::kHalf, a.c.data + (size_t)at_b * O::kBlock + part * C::kHalf, C::kHalf,
                   &s->full[st]);
      }
      at += r.tiles;
    }
    for (int k = max(0, n - stages); k < n; ++k) mbar_wait_drain(&s->full[ring0 + k % stages], (k / stages) & 1);
  } else if (warp == 1) {
    // ------------------------------------------------ matrix instructions
    if (lane == 0) {
      int n = 0, pairs = 0, runs = 0;  // tiles, pairs of tiles and blocks of rows so far
      for (int at = g0; at < g1;) {
        int blocks;
        const Kv4Run r = kv4_block_run<ACCOUNT>(a, first, seqs, at, g1, &blocks);
        const int np = (r.tiles + 1) / 2;
        for (int rb = 0; rb < blocks; ++rb, ++runs) {
          const int qb = ACCOUNT ? runs & 1 : 0;
          bool ok = kv4_wait(&s->qfull[qb], (ACCOUNT ? runs >> 1 : runs) & 1, s);
          for (int q = 0; q <= np; ++q) {
            if (q < np) {  // scores of pair q
              const int y = pairs + q, kb = y % C::kKBufs, sb = y % C::kSBufs;
              ok = kv4_wait(&s->kfull[kb], (y / C::kKBufs) & 1, s) && ok;
              if (y >= C::kSBufs) ok = kv4_wait(&s->sread[sb], (y / C::kSBufs - 1) & 1, s) && ok;
              kv4_fence_after();
              if (ok) {
                const uint32_t kaddr = su32(kop + kb * 2 * C::kOperand), qaddr = su32(qop);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                  const uint32_t off = (k >> 2) * (kKv4M * 128) + (k & 3) * 32;
                  const uint64_t kd = kv4_desc(kaddr + off, 0);
                  if (ACCOUNT) kv4_mma_ts(tmem + C::kColS + sb * 128, tmem + C::kColQ + qb * (D / 2) + k * 8, kd, kv4_idesc(128, false), k > 0);
                  else kv4_mma_ss(tmem + C::kColS, kv4_desc(qaddr + off, 0), kd, kv4_idesc(128, false), k > 0);
                }
              }
              kv4_commit(&s->sfull[sb]);
              kv4_commit(&s->kempty[kb]);
              if (ACCOUNT && q + 1 == np) kv4_commit(&s->qdone[qb]);
            }
            if (!ACCOUNT && q > 0) {  // outputs of pair q - 1
              for (int x = 2 * q - 2; x < min(2 * q, r.tiles); ++x) {
                const int y = n + x, b = y & 1;
                ok = kv4_wait(&s->vfull[b], (y >> 1) & 1, s) && ok;
                ok = kv4_wait(&s->pfull[b], (y >> 1) & 1, s) && ok;
                kv4_fence_after();
                if (ok) {
                  const uint32_t vaddr = su32(vop + b * C::kOperand);
#pragma unroll
                  for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int k = 0; k < kKv4N / 16; ++k)
                      kv4_mma_ts(tmem, tmem + C::kColP + b * 64 + part * 32 + k * 8, kv4_desc(vaddr + k * 2048, kKv4N * 128),
                                 kv4_idesc(D, true), x > 0 || part > 0 || k > 0);
                }
                kv4_commit(&s->pvdone[b]);
              }
            }
          }
          n += r.tiles;
          pairs += np;
        }
        at += r.tiles;
      }
      kv4_commit(&s->drained);
      mbar_wait_drain(&s->drained, 0);
    }
  } else if (ACCOUNT && warp >= 12) {
    // ------------------------------------------------ account: queries, a block of rows ahead
    int runs = 0;
    for (int at = g0; at < g1;) {
      int blocks;
      const Kv4Run r = kv4_block_run<ACCOUNT>(a, first, seqs, at, g1, &blocks);
      for (int rb = 0; rb < blocks; ++rb, ++runs) {
        const int qb = runs & 1;
        if (runs >= 2) kv4_wait(&s->qdone[qb], ((runs - 2) >> 1) & 1, s);
        kv4_fence_after();
        kv4_load_queries<D>(a, r, rb * kKv4M + (int)threadIdx.x - 384,
                            tmem + ((uint32_t)((warp - 12) * 32) << 16) + C::kColQ + qb * (D / 2));
        kv4_fence_before();
        mbar_arrive(&s->qfull[qb]);
      }
      at += r.tiles;
    }
  } else if (warp >= 12) {
    // ------------------------------------------------ values: warp 12 + b decodes block b
    const int b = warp - 12, st = C::kKRing;
    int n = 0;
    for (int at = g0; at < g1;) {
      int blocks;
      const Kv4Run r = kv4_block_run<ACCOUNT>(a, first, seqs, at, g1, &blocks);
      for (int x = 0; x < r.tiles; ++x, ++n) {
        const int buf = n & 1;
        kv4_wait(&s->full[st], n & 1, s);
        Kv4BlockValues<D> v;
        v.load(ring + (size_t)st * C::kTile + b * C::kHalf, (s->held[1][n & 15] >> b) & 1, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&s->empty[st]);
        if (n >= 2) kv4_wait(&s->pvdone[buf], ((n - 2) >> 1) & 1, s);
        if (wide) v.template store<true>(b, vop + buf * C::kOperand, lane);
        else v.template store<false>(b, vop + buf * C::kOperand, lane);
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&s->vfull[buf]);
      }
      at += r.tiles;
    }
  } else if (warp >= 8) {
    // ------------------------------------------------ keys: warp 8 + b decodes block b
    const int b = warp - 8;
    int n = 0, pairs = 0;
    for (int at = g0; at < g1;) {
      int blocks;
      const Kv4Run r = kv4_block_run<ACCOUNT>(a, first, seqs, at, g1, &blocks);
      for (int rb = 0; rb < blocks; ++rb) {
        for (int x = 0; x < r.tiles; ++x, ++n) {
          const int y = pairs + (x >> 1), kb = y % C::kKBufs, st = n % C::kKRing;
          kv4_wait(&s->full[st], (n / C::kKRing) & 1, s);
          Kv4BlockKeys<D> k;
          k.load(ring + (size_t)st * C::kTile + b * C::kHalf, (s->held[0][n & 15] >> b) & 1, lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(&s->empty[st]);
          if (y >= C::kKBufs) kv4_wait(&s->kempty[kb], (y / C::kKBufs - 1) & 1, s);
          if (wide) k.template store<true>((x & 1) * 4 + b, kop + kb * 2 * C::kOperand, lane);
          else k.template store<false>((x & 1) * 4 + b, kop + kb * 2 * C::kOperand, lane);
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&s->kfull[kb]);
            if (x + 1 == r.tiles && !(x & 1)) mbar_arrive(&s->kfull[kb]);  // a last pair of one tile
          }
        }
        pairs += (r.tiles + 1) / 2;
      }
      at += r.tiles;
    }
  } else if (warp >= 4) {
    // ------------------------------------------------ softmax: a query row per thread
    const int row_in = threadIdx.x - 128, wq = warp - 4;
    const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16);
    const float sc = wide ? a.scale : a.scale * kKv4Up, up = wide ? 1.f : kKv4Up;
    int n = 0, pairs = 0, piece = 0;
    for (int at = g0; at < g1; ++piece) {
      int blocks;
      const Kv4Run r = kv4_block_run<ACCOUNT>(a, first, seqs, at, g1, &blocks);
      const int n_rows = r.m * a.group;
      if (ACCOUNT)
        for (int k = row_in; k < 4 * r.tiles * kKv4N; k += 128) gacc[k] = 0.f;
      if (ACCOUNT) named_bar_sync(2, 128);
      for (int rb = 0; rb < blocks; ++rb) {
        const int row0 = (ACCOUNT ? rb : r.row_tile) * kKv4M, row = row0 + row_in;
        const int tok = min(row, n_rows - 1) / a.group, hq = r.head * a.group + min(row, n_rows - 1) % a.group;
        if (!ACCOUNT) {
          kv4_share_queries<D>(a, r, row0, qop, row_in);
          mbar_arrive(&s->qfull[0]);
        }
        // rows it sees: (low, last]
        const int last = r.len - r.m + tok, low = a.window > 0 ? last - a.window : -1;
        const int tok_max = min(row0 + kKv4M, n_rows) - 1;
        const int last_min = r.len - r.m + row0 / a.group, low_max = a.window > 0 ? r.len - r.m + tok_max / a.group - a.window : -1;
        const float lse = !ACCOUNT ? 0.f
                          : row < n_rows ? __ldcg(a.lse + ((long)r.seq * a.c.kvh + r.head) * a.lse_rows + row) : INFINITY;
        float m = -INFINITY, l = 0.f;
        float factor = sc, ref = 0.f;  // of the exponentials' arguments
        const float fused = ACCOUNT && __any_sync(0xFFFFFFFFu, fabsf(lse) > kKv4FarAccount && fabsf(lse) != INFINITY) ? 1.f : sc;
        for (int x = 0; x < r.tiles; ++x, ++n) {
          const int y = pairs + (x >> 1), sb = y % C::kSBufs;
          kv4_wait(&s->sfull[sb], (y / C::kSBufs) & 1, s);
          kv4_fence_after();
          uint32_t v[64];
          const uint32_t cols = lane_base + C::kColS + sb * 128 + (x & 1) * kKv4N;
          kv4_tld32(cols, v);
          kv4_tld32(cols + 32, v + 32);
          kv4_tld_wait();
          const int j0 = (r.tile + x) * kKv4N;
          const uint32_t have = s->held[0][n & 15];
          kv4_fence_before();
          if ((x & 1) || x + 1 == r.tiles) mbar_arrive(&s->sread[sb]);  // the pair's scores are in registers
          float f[64];
#pragma unroll
          for (int k = 0; k < 64; ++k) f[k] = __uint_as_float(v[k]);
          if (have != 15u || j0 + kKv4N - 1 > last_min || j0 <= low_max) {
#pragma unroll
            for (int k = 0; k < 64; ++k)
              if (j0 + k > last || j0 + k <= low || !((have >> (k >> 4)) & 1)) f[k] = -INFINITY;
          }
          if constexpr (ACCOUNT) {
            kv4_round_far(f, sc, fused);
#pragma unroll
            for (int k = 0; k < 64; ++k) f[k] = kv4_exp2(fmaf(f[k], fused, -lse));
            // each step a lane keeps half of its columns and adds its partner's half of them
#pragma unroll
            for (int o = 16, w = 32; o > 0; o >>= 1, w >>= 1) {
              const bool hi = lane & o;
#pragma unroll
              for (int k = 0; k < w; ++k) {
                const float keep = hi ? f[k + w] : f[k], send = hi ? f[k] : f[k + w];
                f[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
              }
            }
            float* to = gacc + (wq * r.tiles + x) * kKv4N + 2 * lane;  // lane's columns: 2 lane, 2 lane + 1
            to[0] += f[0];
            to[1] += f[1];
          } else {
            float mx = f[0];
#pragma unroll
            for (int k = 1; k < 64; ++k) mx = fmaxf(mx, f[k]);
            const float raw = mx;
            mx = __fmul_rn(mx, sc);
            const bool raise = mx > m + 8.f || (m == -INFINITY && mx > m);
            if (__any_sync(0xFFFFFFFFu, raise)) {  // a row's numbers do not depend on its neighbours'
              const float nm = raise ? mx : m, fac = raise ? kv4_exp2(m - nm) : 1.f;
              m = nm;
              l *= fac;
              if (raise) {
                const bool far = fabsf(m) >= kKv4FarAttention && fabsf(m) != INFINITY;
                factor = far ? kv4_power_below(sc) : sc;
                ref = far ? __fmul_rn(raw, factor) : m;
              }
              if (x > 0) {  // the output so far follows: the previous tile's product has to be in
                kv4_wait(&s->pvdone[(n - 1) & 1], ((n - 1) >> 1) & 1, s);
                kv4_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                  uint32_t u[32];
                  kv4_tld32(lane_base + c, u);
                  kv4_tld_wait();
#pragma unroll
                  for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * fac);
                  kv4_tst32(lane_base + c, u);
                }
                kv4_tst_wait();
              }
            }
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float p0 = kv4_exp2(fmaf(f[2 * k], factor, -ref)), p1 = kv4_exp2(fmaf(f[2 * k + 1], factor, -ref));
              s0 += p0;
              s1 += p1;
              v[k] = as_u32(__floats2bfloat162_rn(p0, p1));
              v[32 + k] = as_u32(__floats2bfloat162_rn(p0 - bf16_lo(v[k]), p1 - bf16_hi(v[k])));
            }
            l += s0 + s1;
            const int pb = n & 1;
            if (n >= 2) {  // the weights before the previous tile's have been used
              kv4_wait(&s->pvdone[pb], ((n - 2) >> 1) & 1, s);
              kv4_fence_after();
            }
            kv4_tst32(lane_base + C::kColP + pb * 64, v);
            kv4_tst32(lane_base + C::kColP + pb * 64 + 32, v + 32);
            kv4_tst_wait();
            kv4_fence_before();
            mbar_arrive(&s->pfull[pb]);
          }
        }
        pairs += (r.tiles + 1) / 2;
        if constexpr (!ACCOUNT) {
          // ---- the run's output row
          kv4_wait(&s->pvdone[(n - 1) & 1], ((n - 1) >> 1) & 1, s);
          kv4_fence_after();
          const bool whole = r.whole;
          const float inv = (whole ? (l != 0.f ? 1.f / l : 0.f) : 1.f) * up;
          const long slot_p = (long)blockIdx.x * 2 + (piece ? 1 : 0);
          float4* part = a.part_o + slot_p * (D / 4) * kKv4M + row_in;  // [D / 4][128 rows]
          const long o0 = (long)r.seq * a.out.seq + (long)tok * a.out.row + (long)hq * a.out.head;
#pragma unroll 1
          for (int c = 0; c < D; c += 64) {
            uint32_t u[64];
            kv4_tld32(lane_base + c, u);
            kv4_tld32(lane_base + c + 32, u + 32);
            kv4_tld_wait();
            float f[64];
#pragma unroll
            for (int k = 0; k < 64; ++k) f[k] = __uint_as_float(u[k]) * inv;
            if (!whole) {
#pragma unroll
              for (int k = 0; k < 16; ++k) part[(c / 4 + k) * kKv4M] = make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
            } else if (row < n_rows) {
#pragma unroll
              for (int k = 0; k < 4; ++k) kv4_store16(a.out, o0 + c + 16 * k, f + 16 * k);
            }
          }
          if (!whole) a.part_ml[slot_p * kKv4M + row_in] = make_float2(m, l);
          else a.lse[((long)r.seq * a.c.kvh + r.head) * a.lse_rows + row] = kv4_lse(make_float2(m, l));
          kv4_fence_before();
        }
      }
      if constexpr (ACCOUNT) {
        named_bar_sync(2, 128);
        const int keys = r.tiles * kKv4N;
        for (int k = row_in; k < keys; k += 128) {
          const int j = r.tile * kKv4N + k;
          if (j >= r.len) continue;
          const long at_b = kv4_block(a.c, r.slot, r.head, j / kKv4Block);
          if (at_b >= 0)
            a.c.weight[at_b * kKv4Block + j % kKv4Block] += (gacc[k] + gacc[keys + k]) + (gacc[2 * keys + k] + gacc[3 * keys + k]);
        }
        named_bar_sync(2, 128);
      }
      at += r.tiles;
    }
  }
  kv4_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && s->abort) set_err(a.c.err, G4_DEV_TIMEOUT);
  if (warp == 1) {
    kv4_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(C::kCols) : "memory");
  }
}

// Joins the parts of shared items, in span order: a thread per row of item blockIdx.x and 16
// numbers of it, blockIdx.y counting those.  Also the zeros of rows that no tile reaches.
template <int D>
__global__ void __launch_bounds__(128) kv4_block_join_kernel(const __grid_constant__ Kv4AttendArgs a, int ctas) {
  extern __shared__ __align__(16) uint8_t kv4_raw[];
  int4* seqs = reinterpret_cast<int4*>(kv4_raw);
  int* first = reinterpret_cast<int*>(seqs + a.n_seq);
  const int item = blockIdx.x, per_seq = a.c.kvh * a.row_tiles, tid = threadIdx.x;
  const int i = item / per_seq, x = item % per_seq, head = x / a.row_tiles, rt = x % a.row_tiles;
  kv4_plan<kKv4N>(a, first, seqs, first + a.n_seq + 2, false);  // inputs of the first launch too: read before it ends
  const int m = seqs[i].z, n = seqs[i].w, n_rows = m * a.group;
  const int span = kv4_span(a, first, ctas), t0 = first[i] + n * x;
  const int c0 = (unsigned)t0 / (unsigned)span, c1 = n ? (int)((unsigned)(t0 + n - 1) / (unsigned)span) : c0 - 1;
  pdl_wait();
  pdl_trigger();
  if (x == 0 && blockIdx.y == 0) kv4_zero_rows<D>(a, first, seqs, i, a.n_seq, tid, 128);
  if (c1 <= c0) return;
  const int row = rt * kKv4M + tid, e = blockIdx.y * 16;
  if (row >= n_rows) return;
  float2 ml = make_float2(-INFINITY, 0.f);
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) kv4_merge_ml(ml, __ldcg(&a.part_ml[kv4_part(c, t0, span) * kKv4M + tid]));
  const float Z = ml.x == -INFINITY ? 0.f : ml.x, inv = ml.y != 0.f ? 1.f / ml.y : 0.f;
  float v[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) v[q] = 0.f;
#pragma unroll 2
  for (int c = c0; c <= c1; ++c) {
    const long p = kv4_part(c, t0, span);
    const float f = kv4_exp2(__ldcg(&a.part_ml[p * kKv4M + tid].x) - Z);
    const float4* o = a.part_o + (p * (D / 4) + e / 4) * kKv4M + tid;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 u = __ldcg(o + q * kKv4M);
      v[4 * q] += f * u.x;
      v[4 * q + 1] += f * u.y;
      v[4 * q + 2] += f * u.z;
      v[4 * q + 3] += f * u.w;
    }
  }
#pragma unroll
  for (int q = 0; q < 16; ++q) v[q] *= inv;
  const int tok = row / a.group, hq = head * a.group + row % a.group;
  kv4_store16(a.out, (long)i * a.out.seq + (long)tok * a.out.row + (long)hq * a.out.head + e, v);
  if (blockIdx.y == 0) a.lse[((long)i * a.c.kvh + head) * a.lse_rows + row] = kv4_lse(ml);
}

}  // namespace g4
