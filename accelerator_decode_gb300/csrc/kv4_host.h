// What the decode step uses of the 4-bit KV cache (kv4.cu): a layer's cache, the workspace all
// layers share, and the two launches of a layer's attention.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv4_layout.h"

namespace g4 {

// Partial sums and counters of an attention launch (kv4_attend.cuh).
struct Kv4Work {
  float* lse = nullptr;
  float4* part_o = nullptr;
  float2* part_ml = nullptr;
  unsigned* tickets = nullptr;
  int sms = 0, smem_optin = 0;
};
size_t kv4_work_lse(int n_seq, int kvh, int group, int q_len);      // entries
size_t kv4_work_part_rows(int sms);                                // rows of part_ml; part_o: head_dim / 4 each
size_t kv4_work_tickets(int n_seq, int kvh, int group, int q_len);
size_t kv4_cache_bytes(size_t blocks, int kvh, int head_dim);
void kv4_init(int device, int smem_optin);  // kernel attributes, once per device

// The step's q / k / v rows (one KV head) of n sequences at positions[i] of slots[i]:
// q[i] = RoPE(RMSNorm(q_raw) g_q), fp32 [n][nq][D]; own: k = RoPE(RMSNorm(k_raw) g_k) and v are
// coded into row positions[i]; lens[i] = positions[i] + 1 (0, with the error word set, where the
// position or slot is outside the cache).
struct Kv4Step {
  const float* qkv;
  int qkv_stride, nq, own;
  const __nv_bfloat16 *g_q, *g_k;
  float eps;
  const float *rope_cos, *rope_sin;
  const int *slots, *positions;
  float* q;
  int* lens;
};
void kv4_step_rows(const Kv4Cache& c, const Kv4Step& a, int n, cudaStream_t st);
// One query token per sequence over rows 0 .. lens[i] - 1: fp32 [n][nq][D] in and out.
void kv4_step_attend(const Kv4Cache& c, const Kv4Work& w, int n, const int* slots, const int* lens, int nq, float scale,
                     int window, float* q, float* out, int out_stride, cudaStream_t st);

}  // namespace g4
