// Softmax attention over the 4-bit cache (kv4.cuh), and the account of attention weights.
//
//   s_j = scale q . K_j      o = sum_j softmax(s)_j V_j      account_j += sum over (t, head) softmax(s)_j
// for the rows j that query token t sees: j <= len - m + t, and j > len - m + t - window.
#pragma once
#include "kv4.cuh"

namespace g4 {

struct Kv4AttendArgs {
  Kv4Cache c;
  const int *slots, *lens, *q_lens;  // q_lens may be NULL
  int q_len, heads, group;           // group: query heads per KV head
  float scale;
  int window, accumulate;
  Kv4Dense q, out;
  float* lse;                        // [n_seq][q_len][heads], log2 of the softmax's sum
};

// Sequence i's slot, rows and query tokens; false (uniform over the block) when it is skipped.
__device__ __forceinline__ bool kv4_seq(const Kv4AttendArgs& a, int i, int* slot, int* len, int* m) {
  *slot = __ldg(a.slots + i);
  *len = __ldg(a.lens + i);
  *m = a.q_lens ? __ldg(a.q_lens + i) : a.q_len;
  int bad = 0;
  if (*slot < 0 || *slot >= a.c.n_slots) bad = G4_DEV_BAD_SLOT;
  else if (*len < 0 || *len > a.c.capacity || *m < 0 || *m > a.q_len) bad = G4_DEV_BAD_POSITION;
  if (a.accumulate && kv4_repeated(a.slots, i, *slot)) bad |= G4_DEV_BAD_SLOT;
  if (bad && threadIdx.x == 0) set_err(a.c.err, bad);
  return bad == 0;
}

constexpr int kKv4AttThreads = 128;

// Octet o of a key / value row as fp32.
template <int D>
__device__ __forceinline__ void kv4_k8(const uint8_t* blk, int r, int o, float (&v)[8]) {
  using O = Kv4Off<D>;
  const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(blk + O::k_word(r, o)));
  const uint32_t s = 0x10001u * __ldg(reinterpret_cast<const uint16_t*>(blk + O::k_scale(r, o >> 2)));
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t x = kv4_pair(w >> (4 * p), s);
    v[2 * p] = bf16_lo(x);
    v[2 * p + 1] = bf16_hi(x);
  }
}
template <int D>
__device__ __forceinline__ void kv4_v8(const uint8_t* blk, int r, int o, float (&v)[8]) {
  using O = Kv4Off<D>;
  const uint32_t s = 0x10001u * __ldg(reinterpret_cast<const uint16_t*>(blk + O::v_scale(r, o >> 2)));
  uint32_t w[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) w[u] = __ldg(reinterpret_cast<const uint16_t*>(blk + O::v_half(r, 2 * o + u)));
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t x = kv4_pair((w[0] | (w[1] << 16)) >> (4 * p), s);
    v[p] = bf16_lo(x);
    v[4 + p] = bf16_hi(x);
  }
}

// One CTA per (query token and head, sequence); a warp takes every fourth key, its lanes the
// octets of the row, with a running maximum and sum per warp.
template <int D>
__global__ void __launch_bounds__(kKv4AttThreads) kv4_attend_kernel(const Kv4AttendArgs a) {
  using O = Kv4Off<D>;
  constexpr int OL = D > 256 ? D / 256 : 1;  // octets per lane
  __shared__ float sm[4], sl[4], so[4][D];
  const int i = blockIdx.y, t = blockIdx.x / a.heads, hq = blockIdx.x % a.heads, h = hq / a.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  int slot, len, m;
  const bool ok = kv4_seq(a, i, &slot, &len, &m);
  if (ok && t >= m) return;
  const int row = ok ? len - m + t : -1;
  const int lo = a.window > 0 ? max(0, row - a.window + 1) : 0;
  float q[OL][8], acc[OL][8], mx = -INFINITY, sum = 0.f;
#pragma unroll
  for (int e = 0; e < OL; ++e) {
    const int o = lane + 32 * e;
    if (o < D / 8) kv4_load8(a.q, i * a.q.seq + t * a.q.row + hq * a.q.head + 8 * o, q[e]);
    else
#pragma unroll
      for (int x = 0; x < 8; ++x) q[e][x] = 0.f;
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[e][x] = 0.f;
  }
  for (int j = lo + warp; j <= row; j += 4) {
    const long b = kv4_block(a.c, slot, h, j / kKv4Block);
    if (b < 0) {
      if (lane == 0) set_err(a.c.err, G4_DEV_BAD_POSITION);
      continue;
    }
    const uint8_t* blk = a.c.data + (size_t)b * O::kBlock;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < OL; ++e) {
      const int o = lane + 32 * e;
      if (o < D / 8) {
        float k[8];
        kv4_k8<D>(blk, j % kKv4Block, o, k);
#pragma unroll
        for (int x = 0; x < 8; ++x) s += q[e][x] * k[x];
      }
    }
    s = warp_sum(s) * a.scale * 1.4426950408889634f;
    const float mn = fmaxf(mx, s), al = exp2f(mx - mn), p = exp2f(s - mn);
    mx = mn;
    sum = sum * al + p;
#pragma unroll
    for (int e = 0; e < OL; ++e) {
      const int o = lane + 32 * e;
      if (o < D / 8) {
        float v[8];
        kv4_v8<D>(blk, j % kKv4Block, o, v);
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[e][x] = acc[e][x] * al + p * v[x];
      }
    }
  }
  if (lane == 0) { sm[warp] = mx; sl[warp] = sum; }
#pragma unroll
  for (int e = 0; e < OL; ++e)
    if (lane + 32 * e < D / 8)
#pragma unroll
      for (int x = 0; x < 8; ++x) so[warp][(lane + 32 * e) * 8 + x] = acc[e][x];
  __syncthreads();
  const float mm = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float w[4], l = 0.f;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    w[x] = sl[x] > 0.f ? exp2f(sm[x] - mm) : (sl[x] != sl[x] ? sl[x] : 0.f);
    l += w[x] * sl[x];
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  for (int o = threadIdx.x; o < D / 8; o += kKv4AttThreads) {
    float v[8];
#pragma unroll
    for (int x = 0; x < 8; ++x)
      v[x] = (w[0] * so[0][8 * o + x] + w[1] * so[1][8 * o + x] + w[2] * so[2][8 * o + x] + w[3] * so[3][8 * o + x]) * inv;
    kv4_store8(a.out, i * a.out.seq + t * a.out.row + hq * a.out.head + 8 * o, v);
  }
  if (threadIdx.x == 0) a.lse[((size_t)i * a.q_len + t) * a.heads + hq] = l != 0.f ? mm + log2f(l) : INFINITY;
}

// A warp per row of (sequence, KV head): the weights it received, recomputed from the scores.
template <int D>
__global__ void __launch_bounds__(kKv4AttThreads) kv4_gain_kernel(const Kv4AttendArgs a) {
  using O = Kv4Off<D>;
  constexpr int OL = D > 256 ? D / 256 : 1;
  const int i = blockIdx.y, h = blockIdx.z, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  int slot, len, m;
  if (!kv4_seq(a, i, &slot, &len, &m)) return;
  for (int j = blockIdx.x * 4 + warp; j < len; j += 4 * gridDim.x) {
    const long b = kv4_block(a.c, slot, h, j / kKv4Block);
    if (b < 0) continue;
    const uint8_t* blk = a.c.data + (size_t)b * O::kBlock;
    float k[OL][8], gain = 0.f;
#pragma unroll
    for (int e = 0; e < OL; ++e)
      if (lane + 32 * e < D / 8) kv4_k8<D>(blk, j % kKv4Block, lane + 32 * e, k[e]);
    for (int t = max(0, j - (len - m)); t < m; ++t)
      for (int g = 0; g < a.group; ++g) {
        const int hq = h * a.group + g;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < OL; ++e) {
          const int o = lane + 32 * e;
          if (o < D / 8) {
            float q[8];
            kv4_load8(a.q, i * a.q.seq + t * a.q.row + hq * a.q.head + 8 * o, q);
#pragma unroll
            for (int x = 0; x < 8; ++x) s += q[x] * k[e][x];
          }
        }
        s = warp_sum(s) * a.scale * 1.4426950408889634f;
        gain += exp2f(s - __ldcg(a.lse + ((size_t)i * a.q_len + t) * a.heads + hq));
      }
    if (lane == 0) a.c.weight[b * kKv4Block + j % kKv4Block] += gain;
  }
}

}  // namespace g4
