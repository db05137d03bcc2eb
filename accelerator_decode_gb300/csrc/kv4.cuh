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
#include "kv4_layout.h"

namespace g4 {

// ------------------------------------------------------------------------- dense rows
// Element type and strides (in elements) of a dense [n_seq][rows][heads][D] tensor.
struct Kv4Dense {
  void* p;
  long seq, row, head;
  int dtype;  // G4_DT_*
  int vec;    // base and strides allow 16-byte accesses of whole octets
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

// -------------------------------------------------------------------------- one group
// Scale of a group from its largest magnitude: one fp32 product (an IEEE division costs about
// ten instructions and buys nothing: any scale this near serves the codes as well).  The
// largest scale whose 7-fold is still a finite bf16 bounds it.
__device__ __forceinline__ __nv_bfloat16 kv4_scale(float amax) {
  return __float2bfloat16_rn(fminf(__fmul_rn(amax, 1.f / 7.f), 4.8301e37f));
}
// Code of x under scale s: round-half-even(x / s) clipped to +-7, exactly.  A quotient in 32
// bits may round onto a border (c + 1/2) s from either side, so a first guess is corrected
// against the borders themselves: (c + 1/2) has 4 significant bits and s has 8, so their
// product is exact.
__device__ __forceinline__ int kv4_code(float x, float s, float up, float inv) {
  const float a = fabsf(x);
  float c = fminf(rintf(a * up * inv), 7.f);
  const float lo = (c - 0.5f) * s, hi = (c + 0.5f) * s;
  const bool odd = ((int)c) & 1;
  if (a > hi || (a == hi && odd)) c += 1.f;
  else if (a < lo || (a == lo && odd)) c -= 1.f;
  const int k = (int)fminf(fmaxf(c, 0.f), 7.f);
  return x < 0.f ? -k : k;
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
  const int* positions;               // append: [n_seq][kvh][n_rows] or NULL (row index)
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

// ------------------------------------------------------------------------------ append
// A thread codes one octet (eight numbers) of a row's key and value; the four lanes of a group
// share their largest magnitude.
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
    const float s = bf16f(sb);
    wide |= s > 0.f && !(s >= kKv4Narrow && s <= kKv4Wide);
    const float up = s < 1e-30f ? 0x1p100f : 1.f;  // keeps the reciprocal of a tiny scale finite
    const float inv = s > 0.f ? 1.f / (s * up) : 0.f;
    uint32_t n[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) n[e] = s > 0.f ? (uint32_t)(kv4_code(v[e], s, up, inv) + 8) : 8u;
    if (b >= 0) {
      if (kv == 0) {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) w |= n[e] << ((e >> 1) * 4 + (e & 1) * 16);
        *reinterpret_cast<uint32_t*>(blk + O::k_word(r, o)) = w;
        if ((o & 3) == 0) *reinterpret_cast<__nv_bfloat16*>(blk + O::k_scale(r, o >> 2)) = sb;
      } else {
#pragma unroll
        for (int u = 0; u < 2; ++u)
          *reinterpret_cast<uint16_t*>(blk + O::v_half(r, 2 * o + u)) =
              (uint16_t)(n[4 * u] | (n[4 * u + 1] << 4) | (n[4 * u + 2] << 8) | (n[4 * u + 3] << 12));
        if ((o & 3) == 0) *reinterpret_cast<__nv_bfloat16*>(blk + O::v_scale(r, o >> 2)) = sb;
      }
    }
  }
  if (odd_value) set_err(a.c.err, G4_DEV_BAD_VALUE);
  if (wide) *a.c.wide = 1;
  if (o == 0 && a.c.pos && b >= 0) {
    const size_t at = ((size_t)i * a.c.kvh + h) * a.n_rows + t;
    a.c.pos[b * kKv4Block + r] = a.positions ? __ldcg(a.positions + at) : row;
    a.c.weight[b * kKv4Block + r] = a.weights ? __ldcg(a.weights + at) : 0.f;
  }
}

// -------------------------------------------------------------------------------- read
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

// ------------------------------------------------------------------------------- evict
// One CTA per (sequence, KV head).  Rows are ranked by a 33-bit key: safe rows first, then the
// weight's bits mapped to an unsigned order (NaN lowest, -0 as +0); `budget`-th largest key by
// counting digits from the top (8 bits a pass), ties broken by the lowest row.
struct Kv4EvictArgs {
  Kv4Cache c;
  const int *slots, *lens;
  int budget, recent;
  int* new_lens;
  int* holes;   // scratch [n_seq][kvh][budget]: rows below the budget that go
  int* movers;  // and the kept rows from beyond it that take their places
  int* n_moves; // [n_seq][kvh]
};

__device__ __forceinline__ uint32_t kv4_rank_bits(float w) {
  if (w != w) return 0u;
  if (w == 0.f) w = 0.f;
  const uint32_t u = __float_as_uint(w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;  // -inf maps to 0x007FFFFF, above NaN's 0
}

constexpr int kKv4EvictThreads = 512;

// Exclusive prefix of one int per thread over the block; *total gets the sum.
__device__ __forceinline__ int kv4_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int base = 0, sum = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < warp) base += warp_sums[w];
    sum += warp_sums[w];
  }
  *total = sum;
  return base + x - v;
}

__global__ void __launch_bounds__(kKv4EvictThreads) kv4_select_kernel(const Kv4EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int sums[32];
  __shared__ int sh_newest, sh_digit, sh_above;
  const int i = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const int slot = __ldcg(a.slots + i), len = __ldcg(a.lens + i);
  int* n_moves = a.n_moves + (size_t)i * a.c.kvh + h;
  int bad = 0;
  if (slot < 0 || slot >= a.c.n_slots) bad = G4_DEV_BAD_SLOT;
  else if (len < 0 || len > a.c.capacity) bad = G4_DEV_BAD_POSITION;
  if (kv4_repeated(a.slots, i, slot)) bad |= G4_DEV_BAD_SLOT;
  if (!bad) {  // every page of the rows is there: a row without one cannot be moved
    int miss = 0;
    const int nb = (len + kKv4Block - 1) / kKv4Block;
    for (int b = tid; b < nb; b += blockDim.x) miss |= kv4_block(a.c, slot, h, b) < 0;
    if (__syncthreads_or(miss)) bad = G4_DEV_BAD_POSITION;
  }
  if (bad) {
    if (tid == 0) {
      set_err(a.c.err, bad);
      *n_moves = 0;
      if (h == 0) a.new_lens[i] = len;
    }
    return;
  }
  if (tid == 0 && h == 0) a.new_lens[i] = min(len, a.budget);
  if (len <= a.budget) {
    if (tid == 0) *n_moves = 0;
    return;
  }
  auto at = [&](int r) { return kv4_block(a.c, slot, h, r / kKv4Block) * kKv4Block + r % kKv4Block; };
  // newest position
  if (tid == 0) sh_newest = INT_MIN;
  __syncthreads();
  int newest = INT_MIN;
  for (int r = tid; r < len; r += blockDim.x) newest = max(newest, a.c.pos[at(r)]);
  atomicMax(&sh_newest, newest);
  __syncthreads();
  const long oldest_safe = (long)sh_newest - a.recent;  // safe: position > this
  auto key = [&](int r) {
    const long x = at(r);
    return ((unsigned long long)((long)a.c.pos[x] > oldest_safe) << 32) | kv4_rank_bits(a.c.weight[x]);
  };
  // the budget-th largest key
  unsigned long long prefix = 0;
  int want = a.budget;  // rows still to take among those that share the prefix
  for (int shift = 32; shift >= 0; shift -= 8) {
    for (int b = tid; b < 256; b += blockDim.x) hist[b] = 0;
    __syncthreads();
    for (int r = tid; r < len; r += blockDim.x) {
      const unsigned long long k = key(r);
      if ((k >> shift >> 8) == (prefix >> shift >> 8)) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int above = 0, dgt = 255;
      for (; dgt > 0 && above + hist[dgt] < want; --dgt) above += hist[dgt];
      sh_digit = dgt;
      sh_above = above;
    }
    __syncthreads();
    want -= sh_above;
    prefix |= (unsigned long long)sh_digit << shift;
  }
  // rows above the key stay; of those equal to it the first `want` do
  int ties = 0, n_holes = 0, n_movers = 0;
  int* holes = a.holes + ((size_t)i * a.c.kvh + h) * a.budget;
  int* movers = a.movers + ((size_t)i * a.c.kvh + h) * a.budget;
  for (int r0 = 0; r0 < len; r0 += blockDim.x) {
    const int r = r0 + tid;
    const unsigned long long k = r < len ? key(r) : 0;
    int total;
    const bool tie = r < len && k == prefix;
    const int before = ties + kv4_scan(tie, sums, &total);
    ties += total;
    const bool kept = r < len && (k > prefix || (tie && before < want));
    const bool hole = r < a.budget && !kept, mover = r >= a.budget && kept;
    const int hi = n_holes + kv4_scan(hole, sums, &total);
    n_holes += total;
    const int mi = n_movers + kv4_scan(mover, sums, &total);
    n_movers += total;
    if (hole) holes[hi] = r;
    if (mover) movers[mi] = r;
  }
  if (tid == 0) *n_moves = n_holes;
}

// Row movers[m] -> row holes[m] of every (sequence, KV head).  Sources lie at or beyond the
// budget and destinations below it, so no move reads what another one writes.  A thread moves
// one octet of the key and of the value.
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
    const int src = __ldcg(a.movers + ih * a.budget + m), dst = __ldcg(a.holes + ih * a.budget + m);
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
