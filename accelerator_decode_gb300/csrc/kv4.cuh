// A KV cache held in 4 bits: layout, coding rows in, giving rows back, evicting rows.
//
// A row of one KV head is a key and a value of D numbers.  Each group of 32 numbers is held as
// signed 4-bit codes under one bf16 scale, the convention of the W4A16 weights:
//   s = bf16(max|x| * (1/7))     c = round-half-even(x / s) clipped to +-7     value = bf16(c * s)
// (1/7 and its product in fp32: a group whose exact quotient lies within an fp32 rounding of the
// middle between two bf16 numbers, about one in 100,000, may take the other one as its scale)
// so a row takes 2 (D/2 + D/16) bytes (D = 256: 288, against 1,024 in bf16 and 520 in int8).
// Every value is finite by construction (append replaces what is not finite), so a row that a
// mask hides can be multiplied by a zero weight without turning the sum into a NaN.
#pragma once
#include <cuda_fp16.h>
#include <limits.h>

#include "common.cuh"
#include "kv4_host.h"
#include "kv4_layout.h"

namespace g4 {

// ------------------------------------------------------------------------- dense rows
// Element type and strides (in elements) of a dense [n_seq][rows][heads][D] tensor.
struct Kv4Dense {
  void* p;
  long seq, row, head;
  int dtype;  // G4_DT_*
  int vec;    // base and strides allow 16-byte (1) or 32-byte (2) accesses of whole octets
};

__device__ __forceinline__ void kv4_load8(const Kv4Dense& x, long off, float (&v)[8]) {
  if (x.dtype == G4_DT_F32) {
    const float* p = reinterpret_cast<const float*>(x.p) + off;
    if (x.vec) {
      const float4 a = __ldcg(reinterpret_cast<const float4*>(p)), b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __ldcg(p + e);
    }
    return;
  }
  uint32_t u[4];
  const uint16_t* p = reinterpret_cast<const uint16_t*>(x.p) + off;
  if (x.vec) {
    const uint4 a = __ldcg(reinterpret_cast<const uint4*>(p));
    u[0] = a.x; u[1] = a.y; u[2] = a.z; u[3] = a.w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = (uint32_t)__ldcg(p + 2 * e) | ((uint32_t)__ldcg(p + 2 * e + 1) << 16);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (x.dtype == G4_DT_BF16) {
      v[2 * e] = bf16_lo(u[e]);
      v[2 * e + 1] = bf16_hi(u[e]);
    } else {
      const __half2 h = *reinterpret_cast<__half2*>(&u[e]);
      v[2 * e] = __low2float(h);
      v[2 * e + 1] = __high2float(h);
    }
  }
}

__device__ __forceinline__ uint32_t kv4_pack2(int dtype, float a, float b) {
  if (dtype == G4_DT_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void kv4_store8(const Kv4Dense& x, long off, const float (&v)[8]) {
  if (x.dtype == G4_DT_F32) {
    float* p = reinterpret_cast<float*>(x.p) + off;
    if (x.vec) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = v[e];
    }
    return;
  }
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = kv4_pack2(x.dtype, v[2 * e], v[2 * e + 1]);
  uint16_t* p = reinterpret_cast<uint16_t*>(x.p) + off;
  if (x.vec) {
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[2 * e] = (uint16_t)u[e];
      p[2 * e + 1] = (uint16_t)(u[e] >> 16);
    }
  }
}

__device__ __forceinline__ void kv4_store4(const Kv4Dense& x, long off, float4 v) {
  if (x.dtype == G4_DT_F32) {
    float* p = reinterpret_cast<float*>(x.p) + off;
    if (x.vec) {
      *reinterpret_cast<float4*>(p) = v;
    } else {
      p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
    }
    return;
  }
  const uint32_t a = kv4_pack2(x.dtype, v.x, v.y), b = kv4_pack2(x.dtype, v.z, v.w);
  uint16_t* p = reinterpret_cast<uint16_t*>(x.p) + off;
  if (x.vec) {
    *reinterpret_cast<uint2*>(p) = make_uint2(a, b);
  } else {
    p[0] = (uint16_t)a; p[1] = (uint16_t)(a >> 16); p[2] = (uint16_t)b; p[3] = (uint16_t)(b >> 16);
  }
}

// Sixteen numbers, in 32-byte accesses where the tensor allows them: a lane then reads or writes
// whole sectors, whatever its neighbours do.
__device__ __forceinline__ void kv4_load32b(const void* p, uint32_t (&u)[8]) {
  asm volatile("ld.global.cg.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
               : "l"(p));
}
__device__ __forceinline__ void kv4_store32b(void* p, const uint32_t (&u)[8]) {
  asm volatile("st.global.v8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};\n" ::"r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]),
               "r"(u[5]), "r"(u[6]), "r"(u[7]), "l"(p)
               : "memory");
}
__device__ __forceinline__ void kv4_load16(const Kv4Dense& x, long off, float* v) {
  uint32_t u[8];
  if (x.vec < 2) {
    kv4_load8(x, off, *reinterpret_cast<float(*)[8]>(v));
    kv4_load8(x, off + 8, *reinterpret_cast<float(*)[8]>(v + 8));
  } else if (x.dtype == G4_DT_F32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      kv4_load32b(reinterpret_cast<const float*>(x.p) + off + 8 * h, u);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[8 * h + e] = __uint_as_float(u[e]);
    }
  } else {
    kv4_load32b(reinterpret_cast<const uint16_t*>(x.p) + off, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (x.dtype == G4_DT_BF16) {
        v[2 * e] = bf16_lo(u[e]);
        v[2 * e + 1] = bf16_hi(u[e]);
      } else {
        const __half2 h = *reinterpret_cast<__half2*>(&u[e]);
        v[2 * e] = __low2float(h);
        v[2 * e + 1] = __high2float(h);
      }
    }
  }
}
__device__ __forceinline__ void kv4_store16(const Kv4Dense& x, long off, const float* v) {
  uint32_t u[8];
  if (x.vec < 2) {
    kv4_store8(x, off, *reinterpret_cast<const float(*)[8]>(v));
    kv4_store8(x, off + 8, *reinterpret_cast<const float(*)[8]>(v + 8));
  } else if (x.dtype == G4_DT_F32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = __float_as_uint(v[8 * h + e]);
      kv4_store32b(reinterpret_cast<float*>(x.p) + off + 8 * h, u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = kv4_pack2(x.dtype, v[2 * e], v[2 * e + 1]);
    kv4_store32b(reinterpret_cast<uint16_t*>(x.p) + off, u);
  }
}

// -------------------------------------------------------------------------- one group
// Scale of a group from its largest magnitude: one fp32 product (an IEEE division costs about
// ten instructions and buys nothing: any scale this near serves the codes as well).  The
// largest scale whose 7-fold is still a finite bf16 bounds it.
__device__ __forceinline__ __nv_bfloat16 kv4_scale(float amax) {
  return __float2bfloat16_rn(fminf(__fmul_rn(amax, 1.f / 7.f), 4.8301e37f));
}
// Codes under scale s: round-half-even(x / s) clipped to +-7, exactly and without a branch.
// q = x (1 / s) is within 1.5 units in the last place of x / s, the remainder x - q s has a few
// significant bits only (s has eight) and comes out of one fma exactly, and a second fma adds
// what it is worth.  The sum meets a border c + 1/2 just where x / s does: beside a border x / s
// is at least ulp(x) / s > 0.501 units of q away from it (24 bits of x, eight of s).  Adding
// 1.5 2^23 then rounds half to even, and leaves the code in the sum's low bits, whose others are
// zero below bit 16: codes are shifted and added as they are.  (A test for nearness to a border
// with a slow path behind it was taken by 1 in 16 warps on bf16 numbers, for their ties.)
// A scale that is tiny or was bounded takes the division (never clipped otherwise: x <= 7.03 s).
struct Kv4Coder {
  float s, inv;
  bool odd;
  __device__ __forceinline__ explicit Kv4Coder(__nv_bfloat16 sb) {
    s = bf16f(sb);
    odd = s > 0.f && !(s >= 0x1p-90f && s < 4.8e37f);
    inv = s > 0.f && !odd ? 1.f / s : 0.f;
  }
  // Four numbers -> their codes + 8 as nibbles, the first in bits 0-3.
  __device__ __forceinline__ uint32_t four(const float* x) const {
    uint32_t u[4];
    if (odd) {
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = far(x[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float q = __fmul_rn(x[e], inv);
        u[e] = __float_as_uint(__fadd_rn(__fmaf_rn(__fmaf_rn(-q, s, x[e]), inv, q), 12582912.f));
      }
    }
    return (u[0] + (u[1] << 4) + (u[2] << 8) + (u[3] << 12) + 0x8888u) & 0xFFFFu;
  }
  __device__ __noinline__ uint32_t far(float x) const {
    const float a = fabsf(x);
    float k = fminf(rintf(a / s), 7.f);  // at most one off
    const float lo = (k - 0.5f) * s, hi = (k + 0.5f) * s;
    const bool one = ((int)k) & 1;
    if (a > hi || (a == hi && one)) k += 1.f;
    else if (a < lo || (a == lo && one)) k -= 1.f;
    return (uint32_t)(int)copysignf(fminf(fmaxf(k, 0.f), 7.f), x);
  }
  // One number: its code + 8.
  __device__ __forceinline__ uint32_t one(float x) const {
    const float v[4] = {x, 0.f, 0.f, 0.f};
    return four(v) & 15u;
  }
};
// A key's word: numbers 2j and 2j + 1 at bits 4j and 16 + 4j.
__device__ __forceinline__ uint32_t kv4_key_word(const Kv4Coder& code, const float* v) {
  const float even[4] = {v[0], v[2], v[4], v[6]}, odd[4] = {v[1], v[3], v[5], v[7]};
  return code.four(even) | code.four(odd) << 16;
}

// Decoding a pair of codes to the bf16 values bf16(c * s).
//
// As the low bits of a bf16 number an integer N of up to 8 bits stands for exactly N 2^-133:
// the subnormals and the first normal binade are one linear scale.  So a nibble n = c + 8 needs
// no exponent patched in, only a mask, wherever it lies in the low byte, and one fma with the
// format's single rounding gives the value, scaled by 2^-64 to keep both factors in range:
//   n 2^-133 * (s 2^69) + (-8 s 2^-64) = (n - 8) s 2^-64          (nibble at bits 0-3)
//   n 2^-129 * (s 2^65) + (-8 s 2^-64)                            (nibble at bits 4-7)
// All three scale factors are exact for 2^-60 <= s <= 2^57.  Two ALU and two bf16 operations a
// pair became 1.25 and 1.  A cache that has ever been given a group outside that range (the
// flag `wide`, set by append) is decoded the plain way: 128 + n under the exponent of 128, minus
// 136, times s.
constexpr float kKv4Up = 18446744073709551616.f;  // 2^64
template <bool WIDE>
struct Kv4Scale {
  uint32_t lo, hi, off;
  __device__ __forceinline__ explicit Kv4Scale(uint32_t s2) {
    if constexpr (WIDE) {
      lo = s2;
    } else {
      lo = as_u32(__hmul2(as_bf162(s2), as_bf162(0x62006200u)));   // s 2^69
      hi = as_u32(__hmul2(as_bf162(s2), as_bf162(0x60006000u)));   // s 2^65
      off = as_u32(__hmul2(as_bf162(s2), as_bf162(0xA100A100u)));  // -8 s 2^-64
    }
  }
  // nibbles J of both halves of w
  template <int J>
  __device__ __forceinline__ uint32_t pair(uint32_t w) const {
    if constexpr (WIDE) {
      const uint32_t x = ((w >> (4 * J)) & 0x000F000Fu) | 0x43004300u;
      return as_u32(__hmul2(__hsub2(as_bf162(x), as_bf162(0x43084308u)), as_bf162(lo)));
    } else {
      const uint32_t x = J >= 2 ? w >> 8 : w;
      return J & 1 ? as_u32(__hfma2(as_bf162(x & 0x00F000F0u), as_bf162(hi), as_bf162(off)))
                   : as_u32(__hfma2(as_bf162(x & 0x000F000Fu), as_bf162(lo), as_bf162(off)));
    }
  }
};
constexpr float kKv4Narrow = 0x1p-60f, kKv4Wide = 0x1p57f;
__device__ __forceinline__ uint32_t kv4_pair(uint32_t w, uint32_t scale2) { return Kv4Scale<true>(scale2).pair<0>(w); }

// Does any earlier entry name the same slot as entry i?  (block-wide; every thread calls it)
__device__ __forceinline__ bool kv4_repeated(const int* slots, int i, int slot) {
  int hit = 0;
  for (int j = threadIdx.x; j < i; j += blockDim.x) hit |= __ldcg(slots + j) == slot;
  return __syncthreads_or(hit) != 0;
}

struct Kv4RowArgs {
  Kv4Cache c;
  const int *slots, *start, *counts;  // counts may be NULL: n_rows each
  int n_rows;
  Kv4Dense k, v;                      // p may be NULL (read)
  const int* positions;               // append: [n_seq][kvh][n_rows] or NULL (on from the newest)
  const float* weights;               // append: same layout, or NULL (0)
  int* positions_out;                 // account
  float* weights_out;
  int zero_rest;                      // read, account: zeros where there is no row
};

// Rows [row0, row0 + count) of sequence i, after its checks; count 0 when it is skipped.
// writes: a slot that an earlier sequence of the call names is skipped too (block-wide).
__device__ __forceinline__ bool kv4_rows_of(const Kv4RowArgs& a, int i, bool writes, int* slot, int* row0, int* count) {
  *slot = __ldcg(a.slots + i);
  *row0 = __ldcg(a.start + i);
  *count = a.counts ? __ldcg(a.counts + i) : a.n_rows;
  int bad = 0;
  if (*slot < 0 || *slot >= a.c.n_slots) bad = G4_DEV_BAD_SLOT;
  else if (*count < 0 || *count > a.n_rows || *row0 < 0 || *row0 > a.c.capacity - *count) bad = G4_DEV_BAD_POSITION;
  if (writes && kv4_repeated(a.slots, i, *slot)) bad |= G4_DEV_BAD_SLOT;
  if (bad && threadIdx.x == 0) set_err(a.c.err, bad);
  return bad == 0;
}

// Positions that append gives by itself: the row's index plus a base per (slot, head), which an
// append at row 0 starts anew and an eviction sets so that the row behind the kept ones follows the
// newest position there was.
__device__ __forceinline__ int kv4_next_position(const Kv4RowArgs& a, int slot, int h, int row0, int row) {
  const long base = row0 ? __ldcg(a.c.base + (size_t)slot * a.c.kvh + h) : 0;
  return (int)min(base + row, (long)INT_MAX);
}
// The base that gives row `rows`, the first behind the held ones, the position `next`.
__device__ __forceinline__ int kv4_base(long next, int rows) { return (int)max(next - rows, (long)INT_MIN); }
// The bases after an append of `count` rows from row0 on: the row behind given positions follows the
// newest of them, or what row0 would have had.  A tracked cache's append has one CTA more per
// sequence for it, so that a long array of positions is read beside the rows (2 x 1,988 positions
// ahead of a CTA's rows made a call 7 us longer).  Nothing else of the call reads a base that this
// changes: the others need one only where no positions are given and row0 > 0.
__device__ __forceinline__ void kv4_set_bases(const Kv4RowArgs& a, int i, int slot, int row0, int count) {
  if (count == 0 || (!a.positions && row0)) return;
  int* base = a.c.base + (size_t)slot * a.c.kvh;
  if (!a.positions) {
    for (int h = threadIdx.x; h < a.c.kvh; h += blockDim.x) base[h] = 0;
    return;
  }
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  const int share = max(1, warps / a.c.kvh);  // warps of a head; those of one head are neighbours
  __shared__ int most[64];
  for (int h = threadIdx.x; h < a.c.kvh; h += blockDim.x) most[h] = INT_MIN;
  __syncthreads();
  for (int h = (threadIdx.x >> 5) / share; h < a.c.kvh; h += warps / share) {
    const int* p = a.positions + ((size_t)i * a.c.kvh + h) * a.n_rows;
    int m = INT_MIN;
#pragma unroll 4
    for (int t = (threadIdx.x >> 5) % share * 32 + lane; t < count; t += 32 * share) m = max(m, __ldcg(p + t));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (lane == 0) atomicMax(&most[h], m);
  }
  __syncthreads();
  for (int h = threadIdx.x; h < a.c.kvh; h += blockDim.x) {
    const long next = max((long)most[h] + 1, row0 ? (long)__ldcg(base + h) + row0 : LONG_MIN);
    base[h] = kv4_base(next, row0 + count);
  }
}

// ------------------------------------------------------------------------------ append
// Two kernels.  In small calls a thread codes one octet (eight numbers) of a row's key and value,
// the four lanes of a group sharing their largest magnitude: short chains, small scattered
// stores.  In large ones a warp codes a whole block of 16 rows in the layout's own order, so that
// codes leave in 8-byte pieces and most groups lie in one lane (kv4_by_blocks has the rule).
// Bound by latency in small calls (one row of eight sequences: 4 us).  Large ones: 16 x 2,100 tokens,
// four heads of 128 in bf16, ragged (67.5 MB, 10 us at the measured copy rate) take 26 us, 2.6 TB/s.
// A number costs 17 instructions, which fill half of the issue slots; the other half waits for loads,
// with 38% of the warps that an SM could hold (72 registers a thread).
constexpr int kKv4RowThreads = 256;

template <int D>
__global__ void __launch_bounds__(kKv4RowThreads) kv4_append_kernel(const Kv4RowArgs a) {
  using O = Kv4Off<D>;
  constexpr int NO = D / 8;
  const int i = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  int slot, row0, count;
  if (!kv4_rows_of(a, i, true, &slot, &row0, &count)) return;
  if (a.c.base && blockIdx.x == gridDim.x - 1) return kv4_set_bases(a, i, slot, row0, count);
  const long unit = ((long)blockIdx.x * kKv4RowThreads + threadIdx.x) / NO;
  const int o = threadIdx.x % NO, h = (int)(unit % a.c.kvh);
  const long t_ = unit / a.c.kvh;
  if (t_ >= count) return;  // whole groups of four lanes leave together (NO is a multiple of 8)
  const int t = (int)t_, row = row0 + t;
  const long b = kv4_block(a.c, slot, h, row / kKv4Block);
  if (b < 0 && o == 0) set_err(a.c.err, G4_DEV_BAD_POSITION);
  uint8_t* blk = a.c.data + (size_t)(b < 0 ? 0 : b) * O::kBlock;
  const int r = row % kKv4Block;
  const unsigned quad = 0xFu << ((threadIdx.x & 31) & ~3);
  bool odd_value = false, wide = false;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const Kv4Dense& x = kv ? a.v : a.k;
    float v[8];
    kv4_load8(x, i * x.seq + t * x.row + h * x.head + 8 * o, v);
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (!(fabsf(v[e]) <= 3.402823466e38f)) {  // NaN counts as 0, an infinity as the largest finite number
        odd_value = true;
        v[e] = v[e] != v[e] ? 0.f : copysignf(3.402823466e38f, v[e]);
      }
      m = fmaxf(m, fabsf(v[e]));
    }
    m = fmaxf(m, __shfl_xor_sync(quad, m, 1));
    m = fmaxf(m, __shfl_xor_sync(quad, m, 2));
    const __nv_bfloat16 sb = kv4_scale(m);
    const Kv4Coder code(sb);
    wide |= code.s > 0.f && !(code.s >= kKv4Narrow && code.s <= kKv4Wide);
    if (b >= 0) {
      if (kv == 0) {
        *reinterpret_cast<uint32_t*>(blk + O::k_word(r, o)) = kv4_key_word(code, v);
        if ((o & 3) == 0) *reinterpret_cast<__nv_bfloat16*>(blk + O::k_scale(r, o >> 2)) = sb;
      } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) *reinterpret_cast<uint16_t*>(blk + O::v_half(r, 2 * o + u)) = (uint16_t)code.four(v + 4 * u);
        if ((o & 3) == 0) *reinterpret_cast<__nv_bfloat16*>(blk + O::v_scale(r, o >> 2)) = sb;
      }
    }
  }
  if (odd_value) set_err(a.c.err, G4_DEV_BAD_VALUE);
  if (wide) *a.c.wide = 1;
  if (o == 0 && a.c.pos && b >= 0) {
    const size_t at = ((size_t)i * a.c.kvh + h) * a.n_rows + t;
    a.c.pos[b * kKv4Block + r] = a.positions ? __ldcg(a.positions + at) : kv4_next_position(a, slot, h, row0, row);
    a.c.weight[b * kKv4Block + r] = a.weights ? __ldcg(a.weights + at) : 0.f;
  }
}

// -------------------------------------------------------------------------------- read
// The inverse, in the same two forms.  Bound by latency in small calls (639 rows of 256: 3.6 us).  Large
// ones: 32 x 2,048 rows, four heads of 128 to fp16 (172 MB) take 31 us, 5.6 TB/s, issue slots 62% busy.
// Eight contexts of up to 8,639 rows of 512 to fp16 (173 MB with the zeros behind the shorter ones)
// take 42 us, 4.2 TB/s: two fifths of the stalls are loads and over a quarter instruction fetches of
// the body unrolled over 512 numbers, with 28% of the warps that an SM could hold (84 registers a thread).
template <int D>
__global__ void __launch_bounds__(kKv4RowThreads) kv4_read_kernel(const Kv4RowArgs a) {
  using O = Kv4Off<D>;
  constexpr int NO = D / 8;
  const int i = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  int slot, row0, count;
  if (!kv4_rows_of(a, i, false, &slot, &row0, &count)) count = 0;
  const long unit = ((long)blockIdx.x * kKv4RowThreads + threadIdx.x) / NO;
  const int o = threadIdx.x % NO, h = (int)(unit % a.c.kvh);
  const long t_ = unit / a.c.kvh;
  if (t_ >= (a.zero_rest ? a.n_rows : count)) return;
  const int t = (int)t_, row = row0 + t, r = row & (kKv4Block - 1);
  long b = -1;
  if (t < count) {
    b = kv4_block(a.c, slot, h, row / kKv4Block);
    if (b < 0 && o == 0) set_err(a.c.err, G4_DEV_BAD_POSITION);
  }
  if (b < 0 && !a.zero_rest) return;
  const uint8_t* blk = a.c.data + (size_t)(b < 0 ? 0 : b) * O::kBlock;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (a.k.p) {
    if (b >= 0) {
      const uint32_t w = __ldcg(reinterpret_cast<const uint32_t*>(blk + O::k_word(r, o)));
      const uint32_t s = 0x10001u * __ldcg(reinterpret_cast<const uint16_t*>(blk + O::k_scale(r, o >> 2)));
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t x = kv4_pair(w >> (4 * p), s);
        v[2 * p] = bf16_lo(x);
        v[2 * p + 1] = bf16_hi(x);
      }
    }
    kv4_store8(a.k, i * a.k.seq + t * a.k.row + h * a.k.head + 8 * o, v);
  }
  if (a.v.p) {
    if (b >= 0) {
      const uint32_t s = 0x10001u * __ldcg(reinterpret_cast<const uint16_t*>(blk + O::v_scale(r, o >> 2)));
      uint32_t w[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) w[u] = __ldcg(reinterpret_cast<const uint16_t*>(blk + O::v_half(r, 2 * o + u)));
      const uint32_t x01 = w[0] | (w[1] << 16);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t x = kv4_pair(x01 >> (4 * p), s);  // number p of both quads
        v[p] = bf16_lo(x);
        v[4 + p] = bf16_hi(x);
      }
    }
    kv4_store8(a.v, i * a.v.seq + t * a.v.row + h * a.v.head + 8 * o, v);
  }
}

// Positions and accumulated weights of rows, [n_seq][kvh][n_rows].
__global__ void __launch_bounds__(kKv4RowThreads) kv4_account_kernel(const Kv4RowArgs a) {
  const int i = blockIdx.y, h = blockIdx.z;
  pdl_wait();
  pdl_trigger();
  int slot, row0, count;
  if (!kv4_rows_of(a, i, false, &slot, &row0, &count)) count = 0;
  const int t = blockIdx.x * kKv4RowThreads + threadIdx.x;
  if (t >= (a.zero_rest ? a.n_rows : count)) return;
  const int row = row0 + t;
  long b = -1;
  if (t < count) {
    b = kv4_block(a.c, slot, h, row / kKv4Block);
    if (b < 0) set_err(a.c.err, G4_DEV_BAD_POSITION);
  }
  if (b < 0 && !a.zero_rest) return;
  const size_t at = ((size_t)i * a.c.kvh + h) * a.n_rows + t;
  if (a.positions_out) a.positions_out[at] = b < 0 ? 0 : __ldcg(a.c.pos + b * kKv4Block + row % kKv4Block);
  if (a.weights_out) a.weights_out[at] = b < 0 ? 0.f : __ldcg(a.c.weight + b * kKv4Block + row % kKv4Block);
}

// ------------------------------------------------------------------ the step's rows
// A warp per query head, and one more for the new key and value: norm and RoPE as the decode
// step's other caches apply them (number lane + 32 e of a row in register e, so a group of 32 is
// one register across the warp).  Bound by latency: two dependent loads, the norm and the stores.
template <int D>
__global__ void __launch_bounds__(32) kv4_step_kernel(const Kv4Cache c, const Kv4Step a) {
  using O = Kv4Off<D>;
  __shared__ uint8_t code_s[2][D];
  const int unit = blockIdx.x, i = blockIdx.y, lane = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const int p = __ldcg(a.positions + i), slot = __ldcg(a.slots + i);
  const bool ok = p >= 0 && p < c.capacity && slot >= 0 && slot < c.n_slots;
  if (unit == 0 && lane == 0) {
    if (p < 0 || p >= c.capacity) set_err(c.err, G4_DEV_BAD_POSITION);
    if (slot < 0 || slot >= c.n_slots) set_err(c.err, G4_DEV_BAD_SLOT);
    a.lens[i] = ok ? p + 1 : 0;
  }
  if (!ok) return;
  const float* raw = a.qkv + (size_t)i * a.qkv_stride + (size_t)unit * D;  // unit nq: the key, the value behind it
  const bool key = unit == a.nq;
  float x[D / 32], v[D / 32], cs[D / 64], sn[D / 64];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {
    x[e] = __ldcg(raw + lane + 32 * e);
    if (key) v[e] = __ldcg(raw + D + lane + 32 * e);
  }
#pragma unroll
  for (int e = 0; e < D / 64; ++e) {
    cs[e] = __ldg(a.rope_cos + (size_t)p * (D / 2) + lane + 32 * e);
    sn[e] = __ldg(a.rope_sin + (size_t)p * (D / 2) + lane + 32 * e);
  }
  const __nv_bfloat16* gain = key ? a.g_k : a.g_q;
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) ss += x[e] * x[e];
  const float den = rms_denom(warp_sum(ss), D, a.eps);
#pragma unroll
  for (int e = 0; e < D / 32; ++e) x[e] = (x[e] / den) * bf16f(gain[lane + 32 * e]);
#pragma unroll
  for (int e = 0; e < D / 64; ++e) {  // RoPE pairs number i with i + D/2
    const float u = x[e], w = x[e + D / 64];
    x[e] = u * cs[e] - w * sn[e];
    x[e + D / 64] = w * cs[e] + u * sn[e];
  }
  if (!key) {
#pragma unroll
    for (int e = 0; e < D / 32; ++e) a.q[((size_t)i * a.nq + unit) * D + lane + 32 * e] = x[e];
    return;
  }
  const long b = kv4_block(c, slot, 0, p / kKv4Block);
  if (b < 0) {
    if (lane == 0) set_err(c.err, G4_DEV_BAD_POSITION);
    return;
  }
  uint8_t* blk = c.data + (size_t)b * O::kBlock;
  const int r = p % kKv4Block;
  bool odd_value = false, wide = false;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      float y = kv ? v[e] : x[e];
      if (!(fabsf(y) <= 3.402823466e38f)) {
        odd_value = true;
        y = y != y ? 0.f : copysignf(3.402823466e38f, y);
      }
      const __nv_bfloat16 sb = kv4_scale(warp_max(fabsf(y)));
      const Kv4Coder code(sb);
      wide |= code.s > 0.f && !(code.s >= kKv4Narrow && code.s <= kKv4Wide);
      code_s[kv][lane + 32 * e] = (uint8_t)code.one(y);
      if (lane == 0) *reinterpret_cast<__nv_bfloat16*>(blk + (kv ? O::v_scale(r, e) : O::k_scale(r, e))) = sb;
    }
  }
  __syncwarp();
  for (int o = lane; o < D / 8; o += 32) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) w |= (uint32_t)code_s[0][8 * o + e] << ((e >> 1) * 4 + (e & 1) * 16);
    *reinterpret_cast<uint32_t*>(blk + O::k_word(r, o)) = w;
  }
  for (int u = lane; u < D / 4; u += 32) {
    const uint8_t* n = code_s[1] + 4 * u;
    *reinterpret_cast<uint16_t*>(blk + O::v_half(r, u)) = (uint16_t)(n[0] | (n[1] << 4) | (n[2] << 8) | (n[3] << 12));
  }
  if (odd_value) set_err(c.err, G4_DEV_BAD_VALUE);
  if (wide) *c.wide = 1;
}

// ---------------------------------------------------------------------- whole blocks
// A warp per (block of 16 rows, KV head), keys (blockIdx.z 0) and values (1) apart: unit u of
// sequence i is head u % kvh of the block that holds row start + 16 (u / kvh).  live: bit r = row
// r of the block is the call's and its index in the call is below `count`.
constexpr int kKv4BlockWarps = 4;
struct Kv4BlockUnit {
  int slot, row0;       // the sequence's
  int head, row, base;  // first row of the block; the call's index of it (may be negative)
  long at;              // pool index, -1: no page
  unsigned live, rest;  // rows with data; rows of the call without (zero_rest)
};
__device__ __forceinline__ bool kv4_block_unit(const Kv4RowArgs& a, int i, bool writes, Kv4BlockUnit* x) {
  int slot, row0, count;
  if (!kv4_rows_of(a, i, writes, &slot, &row0, &count)) {
    if (!a.zero_rest) return false;
    count = row0 = 0;
  }
  if (writes && a.c.base && blockIdx.x == gridDim.x - 1) {
    if (blockIdx.z == 0) kv4_set_bases(a, i, slot, row0, count);
    return false;
  }
  x->slot = slot;
  x->row0 = row0;
  const int limit = a.zero_rest ? a.n_rows : count;
  const long u = (long)blockIdx.x * kKv4BlockWarps + (threadIdx.x >> 5);
  x->head = (int)(u % a.c.kvh);
  const long b = row0 / kKv4Block + u / a.c.kvh;
  if (b * kKv4Block - row0 >= limit) return false;
  x->row = (int)b * kKv4Block;
  x->base = x->row - row0;
  const int lo = max(0, -x->base), hi = min(kKv4Block, limit - x->base), mid = max(lo, min(kKv4Block, count - x->base));
  const unsigned all = ((1u << hi) - 1u) & ~((1u << lo) - 1u);
  x->live = all & ((1u << mid) - 1u);
  x->at = -1;
  if (x->live) {
    x->at = kv4_block(a.c, slot, x->head, (int)b);
    if (x->at < 0) {
      if ((threadIdx.x & 31) == 0) set_err(a.c.err, G4_DEV_BAD_POSITION);
      x->live = 0;
    }
  }
  x->rest = a.zero_rest ? all & ~x->live : 0u;
  return true;
}

// What a warp's numbers were like: any not finite; any scale outside the narrow range.
struct Kv4Odd {
  bool value = false, wide = false;
};
template <int N>
__device__ __forceinline__ float kv4_amax(float (&v)[N], Kv4Odd& odd) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v[e])));  // a NaN stays
  const bool fine = m <= 3.402823466e38f;
  if (!fine) {  // NaN counts as 0, an infinity as the largest finite number
    odd.value = true;
    m = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (!(fabsf(v[e]) <= 3.402823466e38f)) v[e] = v[e] != v[e] ? 0.f : copysignf(3.402823466e38f, v[e]);
      m = fmaxf(m, fabsf(v[e]));
    }
  }
  return m;
}

template <int D>
__global__ void __launch_bounds__(32 * kKv4BlockWarps) kv4_append_blocks_kernel(const Kv4RowArgs a) {
  using O = Kv4Off<D>;
  const int i = blockIdx.y, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_trigger();
  Kv4BlockUnit x;
  if (!kv4_block_unit(a, i, true, &x) || !x.live) return;
  uint8_t* blk = a.c.data + (size_t)x.at * O::kBlock;
  Kv4Odd odd;
  if (blockIdx.z == 0) {  // ---- keys: rows g and g + 8, numbers [t D/4, (t+1) D/4), 32 (D = 64: 16) at a time
    constexpr int N = D >= 128 ? 32 : 16, NP = N / 16;  // numbers and pieces of a step
    const long from = (long)i * a.k.seq + (long)x.head * a.k.head + t * (D / 4);
#pragma unroll 1
    for (int step = 0; step < 2 * (D / 4 / N); ++step) {  // rolled: the code is fetched anew in every launch
      const int k = step >> 1, half = step & 1, r = g + 8 * half;
      const bool on = (x.live >> r) & 1;
      float v[N];
#pragma unroll
      for (int o = 0; o < N / 16; ++o) {
        if (on) kv4_load16(a.k, from + (long)(x.base + r) * a.k.row + k * N + 16 * o, v + 16 * o);
        else
#pragma unroll
          for (int e = 0; e < 16; ++e) v[16 * o + e] = 0.f;
      }
      float m = kv4_amax(v, odd);
      if (D == 64) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      const __nv_bfloat16 sb = kv4_scale(m);
      const Kv4Coder code(sb);
      odd.wide |= code.s > 0.f && !(code.s >= kKv4Narrow && code.s <= kKv4Wide);
      if (on && (D > 64 || !(t & 1))) *reinterpret_cast<__nv_bfloat16*>(blk + O::k_scale(r, (t * (D / 4) + k * N) / kKv4Group)) = sb;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const uint2 w = make_uint2(kv4_key_word(code, v + 16 * p), kv4_key_word(code, v + 16 * p + 8));
        if (on) *reinterpret_cast<uint2*>(blk + ((k * NP + p) * 32 + lane) * 16 + half * 8) = w;
      }
    }
  }
  if (blockIdx.z == 1) {  // ---- values: rows 2t, 2t + 1, 2t + 8, 2t + 9, numbers [g D/8, (g+1) D/8), N at a time
    constexpr int N = D >= 256 ? 32 : D / 8, NP = N / 8;
    const long from = (long)i * a.v.seq + (long)x.head * a.v.head + g * (D / 8);
#pragma unroll 1
    for (int step = 0; step < 2 * (D / 8 / N); ++step) {
      const int k = step >> 1, pr = step & 1;  // the row pair t or t + 4
      uint32_t w[NP][2] = {};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int r = 2 * t + q + 8 * pr;
        const bool on = (x.live >> r) & 1;
        float v[N];
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = 0.f;
        if (on) {
          const long at = from + (long)(x.base + r) * a.v.row + k * N;
          if constexpr (N == 8) kv4_load8(a.v, at, v);
          else
#pragma unroll
            for (int o = 0; o < N / 16; ++o) kv4_load16(a.v, at + 16 * o, v + 16 * o);
        }
        float m = kv4_amax(v, odd);
        if (D <= 128) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
        if (D == 64) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
        const __nv_bfloat16 sb = kv4_scale(m);
        const Kv4Coder code(sb);
        odd.wide |= code.s > 0.f && !(code.s >= kKv4Narrow && code.s <= kKv4Wide);
#pragma unroll
        for (int o = 0; o < NP; ++o)
#pragma unroll
          for (int e = 0; e < 2; ++e) w[o][e] |= code.four(v + 8 * o + 4 * e) << (16 * q);
        const int n0 = g * (D / 8) + k * N;
        if (on && n0 % kKv4Group == 0) *reinterpret_cast<__nv_bfloat16*>(blk + O::v_scale(r, n0 / kKv4Group)) = sb;
      }
      const unsigned both = (x.live >> (2 * t + 8 * pr)) & 3u;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        uint32_t* to = reinterpret_cast<uint32_t*>(blk + O::kV) + ((k * NP + p) * 32 + lane) * 4 + 2 * pr;
        if (both == 3u) {
          *reinterpret_cast<uint2*>(to) = make_uint2(w[p][0], w[p][1]);
        } else if (both) {
          const int q = both >> 1;  // the one row of the pair that is the call's
#pragma unroll
          for (int e = 0; e < 2; ++e) reinterpret_cast<uint16_t*>(to + e)[q] = (uint16_t)(w[p][e] >> (16 * q));
        }
      }
    }
  }
  if (odd.value) set_err(a.c.err, G4_DEV_BAD_VALUE);
  if (odd.wide) *a.c.wide = 1;
  if (blockIdx.z == 0 && a.c.pos && lane < kKv4Block && ((x.live >> lane) & 1)) {
    const size_t at = ((size_t)i * a.c.kvh + x.head) * a.n_rows + x.base + lane;
    a.c.pos[x.at * kKv4Block + lane] = a.positions ? __ldcg(a.positions + at) : kv4_next_position(a, x.slot, x.head, x.row0, x.row + lane);
    a.c.weight[x.at * kKv4Block + lane] = a.weights ? __ldcg(a.weights + at) : 0.f;
  }
}

template <int D>
__global__ void __launch_bounds__(32 * kKv4BlockWarps) kv4_read_blocks_kernel(const Kv4RowArgs a) {
  using O = Kv4Off<D>;
  const int i = blockIdx.y, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_trigger();
  Kv4BlockUnit x;
  if (!kv4_block_unit(a, i, false, &x)) return;
  const uint8_t* blk = a.c.data + (size_t)(x.at < 0 ? 0 : x.at) * O::kBlock;
  const unsigned any = x.live | x.rest;
  if (blockIdx.z == 0 && a.k.p) {
    uint4 u[D / 64] = {};
    uint32_t s[2][(D / 4 + 31) / 32] = {};
    if (x.live) {
#pragma unroll
      for (int k = 0; k < D / 64; ++k) u[k] = __ldcg(reinterpret_cast<const uint4*>(blk) + k * 32 + lane);
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int k = 0; k < (D / 4 + 31) / 32; ++k)
          s[half][k] = 0x10001u * __ldcg(reinterpret_cast<const uint16_t*>(blk + O::k_scale(g + 8 * half, t * (D / 4) / kKv4Group + k)));
    }
    const long to = (long)i * a.k.seq + (long)x.head * a.k.head + t * (D / 4);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = g + 8 * half;
      if (!((any >> r) & 1)) continue;
      const bool on = (x.live >> r) & 1;
#pragma unroll
      for (int p = 0; p < D / 64; ++p) {
        float v[16];
        const uint32_t c0 = half ? u[p].z : u[p].x, c1 = half ? u[p].w : u[p].y;
        const Kv4Scale<true> sc(s[half][p >> 1]);
        const uint32_t y[8] = {sc.pair<0>(c0), sc.pair<1>(c0), sc.pair<2>(c0), sc.pair<3>(c0),
                               sc.pair<0>(c1), sc.pair<1>(c1), sc.pair<2>(c1), sc.pair<3>(c1)};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[2 * e] = on ? bf16_lo(y[e]) : 0.f;
          v[2 * e + 1] = on ? bf16_hi(y[e]) : 0.f;
        }
        kv4_store16(a.k, to + (long)(x.base + r) * a.k.row + 16 * p, v);
      }
    }
  }
  if (blockIdx.z == 1 && a.v.p) {
    uint4 u[D / 64] = {};
    constexpr int NG = D >= 256 ? D / 256 : 1;
    uint32_t s[2][NG] = {};
    if (x.live) {
#pragma unroll
      for (int k = 0; k < D / 64; ++k) u[k] = __ldcg(reinterpret_cast<const uint4*>(blk + O::kV) + k * 32 + lane);
#pragma unroll
      for (int pr = 0; pr < 2; ++pr)
#pragma unroll
        for (int k = 0; k < NG; ++k)
          s[pr][k] = __ldcg(reinterpret_cast<const uint32_t*>(blk + O::v_scale(2 * t + 8 * pr, g * (D / 8) / kKv4Group + k)));
    }
    const long to = (long)i * a.v.seq + (long)x.head * a.v.head + g * (D / 8);
#pragma unroll
    for (int pr = 0; pr < 2; ++pr) {
      const int r = 2 * t + 8 * pr;
      constexpr int PS = D >= 128 ? 2 : 1;  // pieces stored at a time: 16 numbers, or D = 64's eight
#pragma unroll
      for (int p0 = 0; p0 < D / 64; p0 += PS) {
        float even[8 * PS], odd[8 * PS];
#pragma unroll
        for (int q = 0; q < PS; ++q) {
          const int p = p0 + q;
          const Kv4Scale<true> sc(s[pr][NG > 1 ? p / 4 : 0]);
          const uint32_t c0 = pr ? u[p].z : u[p].x, c1 = pr ? u[p].w : u[p].y;
          const uint32_t y[8] = {sc.pair<0>(c0), sc.pair<1>(c0), sc.pair<2>(c0), sc.pair<3>(c0),
                                 sc.pair<0>(c1), sc.pair<1>(c1), sc.pair<2>(c1), sc.pair<3>(c1)};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            even[8 * q + e] = (x.live >> r) & 1 ? bf16_lo(y[e]) : 0.f;
            odd[8 * q + e] = (x.live >> (r + 1)) & 1 ? bf16_hi(y[e]) : 0.f;
          }
        }
        const long at = to + (long)(x.base + r) * a.v.row + 8 * p0;
        if constexpr (PS == 2) {
          if ((any >> r) & 1) kv4_store16(a.v, at, even);
          if ((any >> (r + 1)) & 1) kv4_store16(a.v, at + a.v.row, odd);
        } else {
          if ((any >> r) & 1) kv4_store8(a.v, at, even);
          if ((any >> (r + 1)) & 1) kv4_store8(a.v, at + a.v.row, odd);
        }
      }
    }
  }
}

// ------------------------------------------------------------------------------- evict
// One CTA per (sequence, KV head).  A row's rank is 32 bits: all ones when it is safe, else its
// weight's bits in an unsigned order (NaN lowest, then -inf; -0 as +0), which stays below.  The
// budget-th largest rank is found by counting digits from the top, 8 bits a pass, with the ranks
// in shared memory; a pass ends the search when the digit's rows are wanted all.  Ties go to the
// lowest rows.  Bound by latency: a handful of passes of about a microsecond over a few KB
// (1,025 rows: 10 us; 2,500: 18 us).  One thread walking the 256 counts, and ranks read anew from
// global memory in each pass, took 35 us at 1,025 rows.
struct Kv4EvictArgs {
  Kv4Cache c;
  const int *slots, *lens;
  int budget, recent;
  int* new_lens;
  int* holes;    // scratch [n_seq][kvh][most]: rows below the budget that go
  int* movers;   // and the kept rows from beyond it that take their places
  int most;      // a slot's moves at the most: half its rows
  int* n_moves;  // [n_seq][kvh]
  int smem_rows; // ranks that fit in shared memory
};

__device__ __forceinline__ uint32_t kv4_rank_bits(float w) {
  if (w != w) return 0u;
  if (w == 0.f) w = 0.f;
  const uint32_t u = __float_as_uint(w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;  // -inf: 0x007FFFFF; +inf: 0xFF800000
}

constexpr int kKv4EvictThreads = 512;
constexpr int kKv4EvictWarps = kKv4EvictThreads / 32;

// RANKS: all ranks of the slot are in shared memory (else they are read anew in each pass).
template <bool RANKS>
__device__ __forceinline__ void kv4_select(const Kv4EvictArgs& a, int i, int h, int slot, int len, uint32_t* ranks) {
  __shared__ int hist[256];
  __shared__ int counts[3][kKv4EvictWarps];
  __shared__ int sh_newest, sh_base, sh_digit, sh_want, sh_all;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto at = [&](int r) { return kv4_block(a.c, slot, h, r / kKv4Block) * kKv4Block + r % kKv4Block; };
  // newest position; the positions wait where the ranks will be
  if (tid == 0) {
    sh_newest = INT_MIN;
    sh_base = __ldcg(a.c.base + (size_t)slot * a.c.kvh + h);
  }
  if (tid < 256) hist[tid] = 0;
  __syncthreads();
  int newest = INT_MIN;
#pragma unroll 4
  for (int r = tid; r < len; r += kKv4EvictThreads) {
    const int p = __ldcg(a.c.pos + at(r));
    if (RANKS) ranks[r] = (uint32_t)p;
    newest = max(newest, p);
  }
  newest = __reduce_max_sync(0xFFFFFFFFu, newest);
  if (lane == 0) atomicMax(&sh_newest, newest);
  __syncthreads();
  const long oldest_safe = (long)sh_newest - a.recent;  // safe: position > this
  auto make = [&](int p, float w) { return (long)p > oldest_safe ? 0xFFFFFFFFu : kv4_rank_bits(w); };
  auto rank = [&](int r) { return RANKS ? ranks[r] : make(__ldcg(a.c.pos + at(r)), __ldcg(a.c.weight + at(r))); };
  // the budget-th largest rank: `prefix` after the passes, of which the first `want` rows stay
  uint32_t prefix = 0, mask = 0;
  int want = a.budget;
  bool all = false;
  for (int shift = 24; shift >= 0 && !all; shift -= 8) {
#pragma unroll 4
    for (int r = tid; r < len; r += kKv4EvictThreads) {
      uint32_t k;
      if (RANKS && shift == 24) {  // a thread turns its own positions into ranks
        k = make((int)ranks[r], __ldcg(a.c.weight + at(r)));
        ranks[r] = k;
      } else {
        k = rank(r);
      }
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {  // lane: digits 8 lane .. 8 lane + 7; rows with a larger digit than the lane's
      int n[8], sum = 0;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        n[x] = hist[8 * lane + x];
        sum += n[x];
      }
      int above = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_down_sync(0xFFFFFFFFu, above, o);
        if (lane + o < 32) above += y;
      }
      above -= sum;
#pragma unroll
      for (int x = 7; x >= 0; --x) {
        if (above < want && above + n[x] >= want) {
          sh_digit = 8 * lane + x;
          sh_want = want - above;
          sh_all = above + n[x] == want;
        }
        above += n[x];
        hist[8 * lane + x] = 0;
      }
    }
    __syncthreads();
    prefix |= (uint32_t)sh_digit << shift;
    mask |= 255u << shift;
    want = sh_want;
    all = sh_all != 0;
  }
  // Rows whose masked rank is larger stay; of the equal ones the first `want`.  A warp owns a run
  // of neighbouring rows: count the equal ones, then holes and movers, then write both lists.
  const int per = ((len + kKv4EvictWarps - 1) / kKv4EvictWarps + 31) / 32 * 32, r0 = warp * per, r1 = min(len, r0 + per);
  int ties = 0;
  for (int r = r0 + lane; r - lane < r1; r += 32) ties += __popc(__ballot_sync(0xFFFFFFFFu, r < r1 && (rank(min(r, len - 1)) & mask) == prefix));
  if (lane == 0) counts[0][warp] = ties;
  __syncthreads();
  int ties_before = 0;
  for (int w = 0; w < warp; ++w) ties_before += counts[0][w];
  const unsigned below = (1u << lane) - 1u;
  int n_holes = 0, n_movers = 0;
  auto walk = [&](auto&& visit) {
    int seen = ties_before;
    for (int r = r0 + lane; r - lane < r1; r += 32) {
      const uint32_t k = rank(min(r, len - 1)) & mask;
      const unsigned tie = __ballot_sync(0xFFFFFFFFu, r < r1 && k == prefix);
      const bool kept = r < r1 && (k > prefix || (k == prefix && seen + __popc(tie & below) < want));
      seen += __popc(tie);
      visit(r, __ballot_sync(0xFFFFFFFFu, r < min(r1, a.budget) && !kept), __ballot_sync(0xFFFFFFFFu, kept && r >= a.budget));
    }
  };
  walk([&](int, unsigned hole, unsigned mover) {
    n_holes += __popc(hole);
    n_movers += __popc(mover);
  });
  if (lane == 0) {
    counts[1][warp] = n_holes;
    counts[2][warp] = n_movers;
  }
  __syncthreads();
  int hole0 = 0, mover0 = 0, total = 0;
  for (int w = 0; w < kKv4EvictWarps; ++w) {
    if (w < warp) {
      hole0 += counts[1][w];
      mover0 += counts[2][w];
    }
    total += counts[1][w];
  }
  int* holes = a.holes + ((size_t)i * a.c.kvh + h) * a.most;
  int* movers = a.movers + ((size_t)i * a.c.kvh + h) * a.most;
  walk([&](int r, unsigned hole, unsigned mover) {
    if ((hole >> lane) & 1) holes[hole0 + __popc(hole & below)] = r;
    if ((mover >> lane) & 1) movers[mover0 + __popc(mover & below)] = r;
    hole0 += __popc(hole);
    mover0 += __popc(mover);
  });
  if (tid == 0) {
    a.n_moves[(size_t)i * a.c.kvh + h] = total;
    // the next row still follows every position there was, the evicted ones too
    a.c.base[(size_t)slot * a.c.kvh + h] = kv4_base(max((long)sh_newest + 1, (long)sh_base + len), a.budget);
  }
}

__global__ void __launch_bounds__(kKv4EvictThreads, 1) kv4_select_kernel(const Kv4EvictArgs a) {
  extern __shared__ uint32_t kv4_ranks[];
  const int i = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const int slot = __ldcg(a.slots + i), len = __ldcg(a.lens + i);
  int* n_moves = a.n_moves + (size_t)i * a.c.kvh + h;
  int bad = 0;
  if (slot < 0 || slot >= a.c.n_slots) bad = G4_DEV_BAD_SLOT;
  else if (len < 0 || len > a.c.capacity) bad = G4_DEV_BAD_POSITION;
  if (kv4_repeated(a.slots, i, slot)) bad |= G4_DEV_BAD_SLOT;
  if (!bad && a.c.table) {  // every page of the rows is there: a row without one cannot be moved
    int miss = 0;
    const int nb = (len + kKv4Block - 1) / kKv4Block;
    for (int b = tid * a.c.bpp; b < nb; b += kKv4EvictThreads * a.c.bpp) miss |= kv4_block(a.c, slot, h, b) < 0;
    if (__syncthreads_or(miss)) bad = G4_DEV_BAD_POSITION;
  }
  if (tid == 0) {
    if (bad) set_err(a.c.err, bad);
    if (h == 0) a.new_lens[i] = bad ? len : min(len, a.budget);
    if (bad || len <= a.budget) *n_moves = 0;
  }
  if (bad || len <= a.budget) return;
  if (len <= a.smem_rows) kv4_select<true>(a, i, h, slot, len, kv4_ranks);
  else kv4_select<false>(a, i, h, slot, len, nullptr);
}

// Row movers[m] -> row holes[m] of every (sequence, KV head).  Sources lie at or beyond the
// budget and destinations below it, so no move reads what another one writes.  A thread moves
// one octet of the key and of the value.  Scattered 2- and 4-byte accesses: 512 rows of 16
// (sequence, head) pairs of 128 take 8.5 us, one row of eight 6.5 us (launch and one dependent
// chain of loads).
template <int D>
__global__ void __launch_bounds__(kKv4RowThreads) kv4_move_kernel(const Kv4EvictArgs a) {
  using O = Kv4Off<D>;
  constexpr int NO = D / 8;
  const int i = blockIdx.y, h = blockIdx.z;
  pdl_wait();
  pdl_trigger();
  const size_t ih = (size_t)i * a.c.kvh + h;
  const int n = __ldcg(a.n_moves + ih), o = threadIdx.x % NO;
  for (int m = (blockIdx.x * kKv4RowThreads + threadIdx.x) / NO; m < n; m += gridDim.x * kKv4RowThreads / NO) {
    const int slot = __ldcg(a.slots + i);
    const int src = __ldcg(a.movers + ih * a.most + m), dst = __ldcg(a.holes + ih * a.most + m);
    const long sb = kv4_block(a.c, slot, h, src / kKv4Block), db = kv4_block(a.c, slot, h, dst / kKv4Block);
    const uint8_t* sp = a.c.data + (size_t)sb * O::kBlock;
    uint8_t* dp = a.c.data + (size_t)db * O::kBlock;
    const int sr = src % kKv4Block, dr = dst % kKv4Block;
    *reinterpret_cast<uint32_t*>(dp + O::k_word(dr, o)) = *reinterpret_cast<const uint32_t*>(sp + O::k_word(sr, o));
#pragma unroll
    for (int u = 0; u < 2; ++u)
      *reinterpret_cast<uint16_t*>(dp + O::v_half(dr, 2 * o + u)) =
          *reinterpret_cast<const uint16_t*>(sp + O::v_half(sr, 2 * o + u));
    if ((o & 3) == 0) {
      *reinterpret_cast<uint16_t*>(dp + O::k_scale(dr, o >> 2)) =
          *reinterpret_cast<const uint16_t*>(sp + O::k_scale(sr, o >> 2));
      *reinterpret_cast<uint16_t*>(dp + O::v_scale(dr, o >> 2)) =
          *reinterpret_cast<const uint16_t*>(sp + O::v_scale(sr, o >> 2));
    }
    if (o == 0) {
      a.c.pos[db * kKv4Block + dr] = a.c.pos[sb * kKv4Block + sr];
      a.c.weight[db * kKv4Block + dr] = a.c.weight[sb * kKv4Block + sr];
    }
  }
}

}  // namespace g4
