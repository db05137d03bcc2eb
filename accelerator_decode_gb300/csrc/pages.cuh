// The page table of a paged cache, kept on the device: pages are given to new rows, shared between
// slots and taken back without the host knowing a length; and the store of rows into the pages.
//
// A pool has n_pages pages of page_size rows.  table[slot][p] names the page of rows
// p * page_size .. of a slot, lens[slot] counts its rows, refs[page] the slots that hold a page, and
// pages that nobody holds lie on a stack: free[0 .. top).  Every result is a function of the arguments
// and that state alone, whatever the order in which threads run.
#pragma once
#include "pages_layout.h"

namespace g4 {

constexpr int kPagesThreads = 1024;
constexpr int kPagesCluster = 8;  // CTAs that truncate or share together

struct PagesShared {
  int slot[kPagesThreads], at[kPagesThreads + 1], from[kPagesThreads], base[kPagesThreads + 1], held[kPagesThreads];
  int seen[kPagesMaxSlots];
  int warp[64];
};

// Inclusive sums of two numbers of every thread of the block; every thread calls it.
__device__ __forceinline__ void pages_scan(int& a, int& b, int* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, a, o), y = __shfl_up_sync(0xFFFFFFFFu, b, o);
    if (lane >= o) a += x, b += y;
  }
  if (lane == 31) red[warp] = a, red[32 + warp] = b;
  __syncthreads();
  if (warp == 0) {
    int x = red[lane], y = red[32 + lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, x, o), v = __shfl_up_sync(0xFFFFFFFFu, y, o);
      if (lane >= o) x += u, y += v;
    }
    red[lane] = x;
    red[32 + lane] = y;
  }
  __syncthreads();
  if (warp) a += red[warp - 1], b += red[31 + warp];
  __syncthreads();
}
// The slot of sequence threadIdx.x, or -1 (with the error word set by `tell`) where it is out of range
// or an earlier sequence of the call names it too.  Every thread calls it.
__device__ __forceinline__ int pages_slot(const Pages& p, const int* slots, int n, int* seen, bool tell) {
  const int i = threadIdx.x;
  if (i < p.n_slots) seen[i] = kPagesThreads;
  __syncthreads();
  int slot = i < n ? __ldcg(slots + i) : -1;
  const bool in = slot >= 0 && slot < p.n_slots;
  if (in) atomicMin(&seen[slot], i);
  __syncthreads();
  if (i < n && (!in || seen[slot] != i)) {
    if (tell) set_err(p.err, G4_DEV_BAD_SLOT);
    slot = -1;
  }
  return in ? slot : -1;
}
// The last entry of at[0 .. n) that is at most e (at[0] = 0, rising).
__device__ __forceinline__ int pages_find(const int* at, int n, int e) {
  int lo = 0, hi = n;  // at[lo] <= e < at[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= e) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct PagesExtend {
  Pages p;
  const int *slots, *counts;
  int n, n_rows;
  int *rows, *offsets, *lens;  // [n_rows], [n + 1], [n]
};

// Every CTA works the whole plan out for itself (a sequence per thread, two sums over the block) and
// writes its part of the rows and of the new pages' names; the last CTA to finish, when all have read
// the old state and the arguments, writes the new state, offsets and lengths.  Latency bounds it: three dependent
// loads and the sums.  With the truncation before it: 64 sequences by 5 rows 10.3 us, 250 sequences by 896 to 1,790 rows (336,195 rows) 15.5 us.
__global__ void __launch_bounds__(kPagesThreads) pages_extend_kernel(const PagesExtend a) {
  __shared__ PagesShared s;
  __shared__ int last;
  const Pages& p = a.p;
  const int i = threadIdx.x;
  const bool tell = blockIdx.x == 0;
  pdl_wait();
  pdl_trigger();
  const int slot = pages_slot(p, a.slots, a.n, s.seen, tell);
  const int top = __ldcg(p.top);
  int places = 0, need = 0, held = 0, old = 0, count = 0;
  bool ok = slot >= 0;
  if (i < a.n) {
    count = __ldcg(a.counts + i);
    if (count >= 0 && count <= p.capacity()) places = count;
    if (ok) {
      held = __ldcg(p.lens + slot);
      ok = count >= 0 && held >= 0 && held <= p.capacity() && count <= p.capacity() - held;
      if (ok && count > 0 && (held & (p.page() - 1))) {  // a page that another slot reads takes no rows
        const int page = __ldcg(p.table + (long)slot * p.max_pages + (held >> p.log_page));
        ok = page >= 0 && page < p.n_pages && __ldcg(p.refs + page) == 1;
      }
      if (!ok && tell) set_err(p.err, G4_DEV_BAD_POSITION);
      if (ok) {
        old = p.pages_of(held);
        need = p.pages_of(held + count) - old;
      }
    }
  }
  int sum = places, upto = need;
  pages_scan(sum, upto, s.warp);
  if (ok && need > 0 && upto > top) {
    ok = false;
    if (tell) set_err(p.err, G4_DEV_NO_PAGES);
  }
  s.slot[i] = ok ? slot : -1;
  s.held[i] = held;
  s.from[i] = old;
  s.at[i + 1] = sum;
  s.base[i + 1] = upto;
  if (i == 0) s.at[0] = s.base[0] = 0;
  __syncthreads();

  // new pages; those of sequences that were passed over for want of pages are all behind the others
  const int fresh = min(s.base[a.n], top), threads = gridDim.x * kPagesThreads, me = blockIdx.x * kPagesThreads + i;
  for (int e = me; e < fresh; e += threads) {
    const int q = pages_find(s.base, a.n, e);
    if (s.slot[q] < 0) continue;
    const int page = __ldcg(p.free + top - 1 - e);
    p.table[(long)s.slot[q] * p.max_pages + s.from[q] + e - s.base[q]] = page;
    if (page >= 0 && page < p.n_pages) p.refs[page] = 1;
  }
  // rows, four at a time
  const int total = s.at[a.n];
  const bool wide = (reinterpret_cast<uintptr_t>(a.rows) & 15) == 0;
  for (long t4 = 4L * me; t4 < a.n_rows; t4 += 4L * threads) {
    const int t0 = (int)t4;
    int r[4] = {-1, -1, -1, -1};
    int q = t0 < total ? pages_find(s.at, a.n, t0) : a.n;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (t4 + k >= total) continue;
      const int t = t0 + k;
      while (t >= s.at[q + 1]) ++q;
      if (s.slot[q] < 0) continue;
      const int row = s.held[q] + t - s.at[q], pg = row >> p.log_page;
      const int page = pg < s.from[q] ? __ldcg(p.table + (long)s.slot[q] * p.max_pages + pg) : __ldcg(p.free + top - 1 - (s.base[q] + pg - s.from[q]));
      r[k] = (page << p.log_page) + (row & (p.page() - 1));
    }
    if (wide && t4 + 4 <= a.n_rows) {
      *reinterpret_cast<int4*>(a.rows + t0) = make_int4(r[0], r[1], r[2], r[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (t4 + k < a.n_rows) a.rows[t4 + k] = r[k];
    }
  }

  if (gridDim.x > 1) {
    __syncthreads();
    if (i == 0) {
      __threadfence();
      last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
      __threadfence();
    }
    __syncthreads();
    if (!last) return;
    if (i == 0) *p.ticket = 0;
  }
  __syncthreads();  // all have read, the arguments too: offsets and new lengths may be written over them
  if (i < a.n) {
    a.offsets[i + 1] = sum;
    a.lens[i] = slot >= 0 ? ok ? held + count : held : 0;
    if (i == 0) a.offsets[0] = 0;
  }
  if (ok) p.lens[slot] = held + count;
  int most = ok && need > 0 ? upto : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
  if ((i & 31) == 0) s.warp[i >> 5] = most;
  __syncthreads();
  if (i < 32) {
    most = s.warp[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    if (i == 0) *p.top = top - most;
  }
}

// Arrives at and waits for the cluster's barrier; global writes before it are seen behind it.
__device__ __forceinline__ void pages_cluster_sync() {
  __threadfence();
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;\n" ::: "memory");
}

struct PagesTruncate {
  Pages p;
  const int *slots, *lens;  // lens NULL: nothing is kept
  int n;
};

// A cluster of CTAs goes over the entries that are let go, in the order of the sequences and their
// rows.  First each lets its page go; where no page was held twice, entry e of E then goes to
// free[top + E - 1 - e], so that the next rows get the pages in the order in which they were held.
// Where pages were held twice, the ones that nobody holds any more go there, in the order of the first
// entry that names them: owner[page] is the lowest such entry, and counting them takes one more pass.
__global__ void __cluster_dims__(kPagesCluster, 1, 1) __launch_bounds__(kPagesThreads) pages_truncate_kernel(const PagesTruncate a) {
  __shared__ PagesShared s;
  const Pages& p = a.p;
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  const bool tell = blockIdx.x == 0;
  pdl_wait();
  pdl_trigger();
  const int slot = pages_slot(p, a.slots, a.n, s.seen, tell);
  const int top = __ldcg(p.top);
  int drop = 0, keep = 0, rows = 0, zero = 0;
  bool ok = slot >= 0;
  if (ok) {
    const int held = __ldcg(p.lens + slot);
    rows = a.lens ? __ldcg(a.lens + i) : 0;
    ok = rows >= 0 && held >= 0 && held <= p.capacity();
    if (!ok && tell) set_err(p.err, G4_DEV_BAD_POSITION);
    ok = ok && rows < held;
    if (ok) {
      keep = p.pages_of(rows);
      drop = p.pages_of(held) - keep;
    }
  }
  int upto = drop;
  pages_scan(upto, zero, s.warp);
  s.slot[i] = slot;
  s.from[i] = keep;
  s.at[i + 1] = upto;
  if (i == 0) s.at[0] = 0;
  __syncthreads();
  const int total = s.at[a.n];  // (sequences that let nothing go have no entries)
  // each warp of the cluster takes a run of entries, 32 at a time
  const int warps = kPagesCluster * kPagesThreads / 32, mine = blockIdx.x * (kPagesThreads / 32) + warp;
  const int per = ((total + warps - 1) / warps + 31) / 32 * 32;
  const int e0 = min(total, mine * per), e1 = min(total, e0 + per);
  auto entry = [&](int e) {
    const int q = pages_find(s.at, a.n, e);
    return p.table + (long)s.slot[q] * p.max_pages + s.from[q] + e - s.at[q];
  };
  int* const twice = p.top + 1;   // whether a page was held twice (or badly)
  int* const counts = p.top + 2;  // [warps] pages that each warp puts back
  constexpr int kEach = 4;  // entries of a lane at a time: their loads, then their atomics, are in flight together
  bool odd = false, bad = false;
  for (int first = e0 + lane; first < e1; first += 32 * kEach) {
    int page[kEach], r[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) page[k] = first + 32 * k < e1 ? __ldcg(entry(first + 32 * k)) : -1;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const bool on = page[k] >= 0 && page[k] < p.n_pages;
      r[k] = on ? atomicSub(p.refs + page[k], 1) : first + 32 * k < e1 ? 0 : 1;
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      odd |= r[k] != 1;
      bad |= r[k] < 1;
    }
  }
  if (bad) set_err(p.err, G4_DEV_BAD_POSITION);
  if (odd) atomicOr(twice, 1);
  pages_cluster_sync();
  const bool some = __ldcg(twice) != 0;
  auto let_go = [&](int e, int page) { return page >= 0 && page < p.n_pages && __ldcg(p.refs + page) == 0 && __ldcg(p.owner + page) == e; };
  int before = 0, all = total;
  if (some) {
    for (int e = e0 + lane; e < e1; e += 32) {
      const int page = __ldcg(entry(e));
      if (page >= 0 && page < p.n_pages && __ldcg(p.refs + page) == 0) atomicMin(p.owner + page, e);
    }
    pages_cluster_sync();
    int n = 0;
    for (int e = e0 + lane; e < e1; e += 32) n += let_go(e, __ldcg(entry(e)));
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (lane == 0) __stcg(counts + mine, n);
    pages_cluster_sync();
    int x = 0, y = 0;
    for (int w = lane; w < warps; w += 32) {
      const int c = __ldcg(counts + w);
      y += c;
      if (w < mine) x += c;
    }
    before = __reduce_add_sync(0xFFFFFFFFu, x);
    all = __reduce_add_sync(0xFFFFFFFFu, y);
  }
  for (int first = e0; first < e1; first += 32 * kEach) {
    int* at[kEach];
    int page[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int e = first + 32 * k + lane;
      at[k] = e < e1 ? entry(e) : nullptr;
      page[k] = at[k] ? __ldcg(at[k]) : -1;
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int e = first + 32 * k + lane;
      const bool back = at[k] && (!some || let_go(e, page[k]));
      const unsigned mask = __ballot_sync(0xFFFFFFFFu, back);
      const int rank = some ? before + __popc(mask & ((1u << lane) - 1)) : e;
      const int to = top + all - 1 - rank;
      if (back && to < p.n_pages) p.free[to] = page[k];
      if (at[k]) *at[k] = -1;
      before += __popc(mask);
    }
  }
  pages_cluster_sync();
  // (owners are looked up behind every entry's last reading of them)
  if (some)
    for (int k = blockIdx.x * kPagesThreads + i; k < all; k += kPagesCluster * kPagesThreads) {
      const int page = __ldcg(p.free + min(top + k, p.n_pages - 1));
      p.owner[page] = 0x7FFFFFFF;
    }
  if (tell) {
    if (ok) p.lens[slot] = rows;
    if (i == 0) {
      *p.top = min(top + all, p.n_pages);
      *twice = 0;
    }
  }
}

struct PagesShare {
  Pages p;
  const int* slots;
  int n, source, n_pages;
};

// Empty slots begin with the source's first n_pages pages.
__global__ void __cluster_dims__(kPagesCluster, 1, 1) __launch_bounds__(kPagesThreads) pages_share_kernel(const PagesShare a) {
  __shared__ PagesShared s;
  const Pages& p = a.p;
  const int i = threadIdx.x;
  const bool tell = blockIdx.x == 0;
  pdl_wait();
  pdl_trigger();
  const int slot = pages_slot(p, a.slots, a.n, s.seen, tell);
  const int held = __ldcg(p.lens + a.source);
  bool ok = slot >= 0;
  if (ok) {
    ok = slot != a.source && __ldcg(p.lens + slot) == 0 && held <= p.capacity() && (held >> p.log_page) >= a.n_pages;
    if (!ok && tell) set_err(p.err, G4_DEV_BAD_POSITION);
  }
  s.slot[i] = ok ? slot : -1;
  __syncthreads();
  const long total = (long)a.n * a.n_pages;
  for (long e = blockIdx.x * kPagesThreads + i; e < total; e += kPagesCluster * kPagesThreads) {
    const int q = (int)(e / a.n_pages), at = (int)(e % a.n_pages);
    if (s.slot[q] < 0) continue;
    const int page = __ldcg(p.table + (long)a.source * p.max_pages + at);
    p.table[(long)s.slot[q] * p.max_pages + at] = page;
    if (page >= 0 && page < p.n_pages) atomicAdd(p.refs + page, 1);
    else set_err(p.err, G4_DEV_BAD_POSITION);
  }
  pages_cluster_sync();
  if (tell && ok) p.lens[slot] = a.n_pages << p.log_page;
}

struct PagesStore {
  Pages p;
  const int* rows;
  int n_rows, kvh, d8, log_d8;       // d8: 16-byte pieces of a row of one head
  const uint16_t *k, *v;
  long k_row, k_head, v_row, v_head;  // strides in elements
  uint16_t *kp, *vp;                  // pools [n_pages][kvh][page][8 d8]
  int vec;
};

constexpr int kPagesStoreThreads = 256;
constexpr int kPagesStoreEach = 4;  // pieces of a thread

// Rows into the pools, 16 bytes of a key and of a value at a time.  HBM bounds it: 33,111 rows of eight
// heads of 128 (271 MB) take 43 us, 0.92 of the measured copy rate.
__global__ void __launch_bounds__(kPagesStoreThreads) pages_store_kernel(const PagesStore a) {
  pdl_wait();
  pdl_trigger();
  const long pieces = (long)a.n_rows * a.kvh * a.d8;
  const long first = (long)blockIdx.x * (kPagesStoreThreads * kPagesStoreEach) + threadIdx.x;
  const long most = (long)a.p.n_pages << a.p.log_page;
  uint4 k[kPagesStoreEach], v[kPagesStoreEach];
  long to[kPagesStoreEach];
#pragma unroll
  for (int x = 0; x < kPagesStoreEach; ++x) {
    const long e = first + (long)x * kPagesStoreThreads;
    to[x] = -1;
    if (e >= pieces) continue;
    const int c = (int)(e & (a.d8 - 1));
    const unsigned hr = (unsigned)(e >> a.log_d8);  // below 2^31 (g4_pages_store)
    const int row = (int)(hr / (unsigned)a.kvh), head = (int)(hr % (unsigned)a.kvh);
    const int at = __ldcg(a.rows + row);
    if (at < 0 || at >= most) {
      if (at != -1) set_err(a.p.err, G4_DEV_BAD_POSITION);
      continue;
    }
    const long page = at >> a.p.log_page, in = at & (a.p.page() - 1);
    to[x] = ((((page * a.kvh + head) << a.p.log_page) + in) << a.log_d8) + c;
    const uint16_t *pk = a.k + (long)row * a.k_row + head * a.k_head + 8 * c, *pv = a.v + (long)row * a.v_row + head * a.v_head + 8 * c;
    if (a.vec) {
      k[x] = __ldcs(reinterpret_cast<const uint4*>(pk));
      v[x] = __ldcs(reinterpret_cast<const uint4*>(pv));
    } else {
      uint32_t w[8];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        w[y] = pk[2 * y] | (uint32_t)pk[2 * y + 1] << 16;
        w[4 + y] = pv[2 * y] | (uint32_t)pv[2 * y + 1] << 16;
      }
      k[x] = make_uint4(w[0], w[1], w[2], w[3]);
      v[x] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
#pragma unroll
  for (int x = 0; x < kPagesStoreEach; ++x)
    if (to[x] >= 0) {
      reinterpret_cast<uint4*>(a.kp)[to[x]] = k[x];
      reinterpret_cast<uint4*>(a.vp)[to[x]] = v[x];
    }
}

}  // namespace g4
