// Index arithmetic of the paged cache, for the kernels and (as plain C++) for
// the host tests: the split of all cached tokens over the CTAs, and where a
// slot's row lies in the page pool.
//
// Tokens are handled in groups of PAGED_GROUP slots; a page holds whole groups,
// so a group's rows of one KV head are contiguous.  A unit is a (sequence, KV
// head); unit (b, h) has ceil(len_b / PAGED_GROUP) groups.  All groups, units in
// order, form one line 0 .. total-1, cut into `parts` ranges of nearly equal
// length: part c takes [part_begin(c), part_begin(c + 1)).  Ragged lengths then
// cost no balance, and a unit is joined from the parts it touches.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define FASA_HD __host__ __device__ __forceinline__
#else
#define FASA_HD inline
#endif

namespace fasa {

constexpr int PAGED_GROUP = 16;         // tokens per group
constexpr int PAGED_PART_GROUPS = 8;    // a part has at least this many groups (while there are as many)
constexpr int PAGED_MAX_PARTS = 320;    // parts the workspace has room for
constexpr int PAGED_MAX_BATCH = 4096;   // the lengths' prefix sums sit in shared memory
constexpr int PAGED_MAX_SLOTS = 524288; // T_cap: the line's positions fit 31 bits

FASA_HD int paged_groups(int len) { return (len + PAGED_GROUP - 1) / PAGED_GROUP; }

// Parts the line is cut into, at most `grid`.
FASA_HD int paged_parts(int total, int grid) {
  const int most = (total + PAGED_PART_GROUPS - 1) / PAGED_PART_GROUPS;
  return most < 1 ? 1 : (most < grid ? most : grid);
}
FASA_HD int paged_part_begin(int total, int parts, int c) { return (int)((long long)total * c / parts); }
// The part that holds position x (0 <= x < total).
FASA_HD int paged_part_of(int total, int parts, int x) {
  return (int)((((long long)x + 1) * parts - 1) / total);
}

// Row (of d elements) of `slot`'s token of KV head h in a pool of pages
// [n_pages, Hkv, page_size, d], the page being page_table's entry; -1 for an
// entry outside the pool.  log2_page: log2(page_size).
FASA_HD long long paged_row(int page, int n_pages, int Hkv, int h, int log2_page, int slot) {
  if (page < 0 || page >= n_pages) return -1;
  return (((long long)page * Hkv + h) << log2_page) + (slot & ((1 << log2_page) - 1));
}

}  // namespace fasa
