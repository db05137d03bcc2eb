// Where the numbers of a 4-bit KV cache lie (plain C++: the host tests compile it too).
//
// Rows are stored in blocks of 16 consecutive rows of one KV head, 18 D bytes each:
//   K codes 8D | K scales D | V codes 8D | V scales D
// with the codes in the order in which the attention kernel's tensor-core fragments take them:
// lane 4g + t of a warp reads whole 16-byte pieces, the warp 512 contiguous bytes (no bank
// conflicts, no shuffles, no transposition in the hot loop).
//   K: lane (g, t) holds rows g and g + 8, numbers [t D/4, (t+1) D/4); word w of a row holds the
//      eight numbers 8w.. of that span.  16-byte piece i = {row g: words 2i, 2i+1; row g+8: same}.
//   V: lane (g, t) holds numbers [g D/8, (g+1) D/8) of the row pairs (2t, 2t+1) and (2t+8,
//      2t+9); word w holds four numbers 4w.. of both rows of a pair (the even row in the low
//      half).  Piece i = {pair t: words 2i, 2i+1; pair t+4: same}.
// In both kinds of word nibble j of the low half and nibble j of the high half belong together
// (numbers 2j and 2j+1 of a key, or number j of two values), so (w >> 4j) & 0x000F000F is a pair
// of codes, ready to become a bf16x2.  A nibble is the code + 8.
//   K scales: [row][group];  V scales: [group][row].
// Blocks of a page (or, in a static cache, of a slot) are contiguous per KV head, so several
// blocks travel in one bulk copy.
#pragma once
#include <stddef.h>
#include <stdint.h>

#ifdef __CUDACC__
#define G4_HD __host__ __device__ __forceinline__
#else
#define G4_HD inline
#endif

namespace g4 {

constexpr int kKv4Block = 16;      // rows per block
constexpr int kKv4Group = 32;      // numbers per scale
constexpr int kKv4MaxSlots = 1024;

struct Kv4Cache {
  uint8_t* data;      // blocks
  int* pos;           // tracked caches: logical position of every row, [page or slot][head][rows]
  float* weight;      // and its accumulated attention weight
  int* base;          // tracked caches: what is added to a row's index for its position, [slot][head]
  const int* table;   // paged: [n_slots][max_pages]; NULL: static
  int log_bpp;        // paged: log2(blocks per page)
  int bpp;            // blocks per page (static: per slot)
  int max_pages, n_pages;
  int n_slots, capacity, kvh, d;
  int* wide;          // 1: a scale outside [2^-60, 2^57] has been stored
  int* err;
};

// Index of block b (of 16 rows) of (slot, head) in the pool, -1 when it has no page.
G4_HD long kv4_block(const Kv4Cache& c, int slot, int head, int b) {
  if (!c.table) return ((long)slot * c.kvh + head) * c.bpp + b;
  const int* at = c.table + (size_t)slot * c.max_pages + (b >> c.log_bpp);
#ifdef __CUDA_ARCH__
  const int pg = __ldcg(at);  // the caller rewrites the table between calls: never from L1
#else
  const int pg = *at;
#endif
  if (pg < 0 || pg >= c.n_pages) return -1;
  return ((long)pg * c.kvh + head) * c.bpp + (b & (c.bpp - 1));
}

// Stages of the attention kernel's ring of key tiles: as many as fit in `room` bytes, two at least and
// four at most, and a multiple of the sets of warps that take tiles in turn (1 or 2).  A warp waits
// for a fill of a stage by the parity of its number, which tells it from the fill before only when
// the warp knows that one to be over.  With a multiple, tile t and tile t - stages belong to the
// same set, which has waited for both; with three stages and two sets the fill before was the
// other set's, and a wait could pass while the copy was still under way.
G4_HD int kv4_ring_stages(long room, int tile, int sets) {
  const long n = room / tile;
  const int stages = n > 4 ? 4 : n < 2 ? 2 : (int)n;
  return stages / sets * sets;
}

// Byte offsets inside a block of D-wide rows.
template <int D>
struct Kv4Off {
  static constexpr int kBlock = 18 * D;
  static constexpr int kKs = 8 * D, kV = 9 * D, kVs = 17 * D;
  // word of row r holding numbers 8 o .. 8 o + 7 of the key
  G4_HD static int k_word(int r, int o) {
    const int t = o / (D / 32), w = o % (D / 32);
    return ((w >> 1) * 32 + (r & 7) * 4 + t) * 16 + ((r >> 3) * 2 + (w & 1)) * 4;
  }
  // 16-bit half-word of row r holding numbers 4 u .. 4 u + 3 of the value
  G4_HD static int v_half(int r, int u) {
    const int g = u / (D / 32), w = u % (D / 32), pair = r >> 1;
    return kV + ((w >> 1) * 32 + g * 4 + (pair & 3)) * 16 + ((pair >> 2) * 2 + (w & 1)) * 4 + (r & 1) * 2;
  }
  G4_HD static int k_scale(int r, int grp) { return kKs + (r * (D / 32) + grp) * 2; }
  G4_HD static int v_scale(int r, int grp) { return kVs + (grp * kKv4Block + r) * 2; }
};

}  // namespace g4
