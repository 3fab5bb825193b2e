// Index arithmetic of the paged cache, for the kernels and (as plain C++) for
// the host tests: the split of all cached tokens over the CTAs, and where a
// slot's row lies in the page pool.
//
// Tokens are handled in groups of PAGED_GROUP slots; a page holds whole groups,
// so a group's rows of one KV head are contiguous.  A unit is a (sequence, KV
// head); unit (b, h) has ceil(len_b / PAGED_GROUP) groups.  All groups, units in
// order, form one line 0 .. total-1, cut into parts, one to a warp; a unit is
// joined from the parts it touches.  The cuts are even in cost: a unit costs
// its groups and PAGED_UNIT_COST more (its query, its output), so that a part
// of many short units takes no longer than one of a long one.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define FASA_HD __host__ __device__ __forceinline__
#else
#define FASA_HD inline
#endif

namespace fasa {

constexpr int PAGED_GROUP = 16;         // tokens per group
// What a unit costs beside its groups, in groups (64 sequences of 0 to 1000 tokens:
// 22.5 us at 0, 17.7 at 1, 17.5 at 2, 18.0 at 4), and the least that a part costs while
// there is as much (one sequence of 1024 tokens: 8.9 us at 4, 7.7 at 2, 7.4 at 1).
constexpr int PAGED_UNIT_COST = 2;
constexpr int PAGED_PART_COST = 1;
constexpr int PAGED_MAX_PARTS = 1280;   // parts the workspace has room for
constexpr int PAGED_MAX_BATCH = 2048;   // the lengths' prefix sums sit in shared memory
constexpr int PAGED_MAX_SLOTS = 262144; // T_cap: the line's positions and costs fit 31 bits

FASA_HD int paged_groups(int len) { return (len + PAGED_GROUP - 1) / PAGED_GROUP; }

// floor(total * c / n), 0 <= c <= n <= 32768.
FASA_HD int cut(int total, int n, int c) {
  const int q = total / n, r = total - q * n;
  return q * c + r * c / n;
}

// Row (of d elements) of `slot`'s token of KV head h in a pool of pages
// [n_pages, Hkv, page_size, d], the page being page_table's entry; -1 for an
// entry outside the pool.  log2_page: log2(page_size).
FASA_HD long long paged_row(int page, int n_pages, int Hkv, int h, int log2_page, int slot) {
  if (page < 0 || page >= n_pages) return -1;
  return (((long long)page * Hkv + h) << log2_page) + (slot & ((1 << log2_page) - 1));
}

// Word b of the line: the groups of one head of the sequences before b (28
// bits: at most 2048 * 16384) and by how many tokens b's last group is short (4
// bits); word B: all sequences' groups.
FASA_HD unsigned paged_word(int before, int len) {
  return (unsigned)before | (unsigned)(paged_groups(len) * PAGED_GROUP - len) << 28;
}

// The line's cuts into n <= PAGED_MAX_PARTS parts, in cost.  (What a cut needs is worked
// out once: a unit's parts are looked up by every warp that reads or joins it.)
struct PagedCuts {
  int n, q, r;
  float part, inv;  // parts per cost, 1 / n

  FASA_HD PagedCuts(int cost, int parts)
      : n(parts), q(cost / (parts > 0 ? parts : 1)), r(cost - q * parts), part(over((float)parts, (float)cost)),
        inv(over(1.f, (float)parts)) {}
  // On the device within 2 steps (2^-22) of a / b.  Rounded to nearest it would be half
  // of one, for 0.1 to 0.2 us of every call.  (b = 0 is an empty line, where nothing is
  // looked up)
  static FASA_HD float over(float a, float b) {
#ifdef __CUDA_ARCH__
    return __fdividef(a, b);
#else
    return b > 0.f ? a / b : 0.f;
#endif
  }
  // Where part c begins, floor(cost * c / n): r c < n^2 and the half behind it are exact in
  // fp32, and the half keeps (r c + 0.5) / n, which is below n, 0.5 / n or more away from
  // every whole number.  inv may be 2^-22 off and the product rounds by 2^-24: 2.5 n 2^-23
  // in all, 3.82e-4 at 1280 parts where 0.5 / n is 3.91e-4.
  FASA_HD int begin(int c) const { return q * c + (int)(((float)(r * c) + 0.5f) * inv); }
};
static_assert(5ll * PAGED_MAX_PARTS * PAGED_MAX_PARTS < 1 << 23, "2.5 n 2^-23 < 0.5 / n: the cuts are exact");

struct PagedLine {
  const unsigned* w;
  int B, Hkv;

  FASA_HD int before(int b) const { return (int)(w[b] & 0x0fffffffu); }
  FASA_HD int groups(int b) const { return before(b + 1) - before(b); }
  FASA_HD int tokens(int b) const { return groups(b) * PAGED_GROUP - (int)(w[b] >> 28); }
  FASA_HD int total() const { return before(B) * Hkv; }
  // The sequence whose units hold position x of the line (0 <= x < total).
  FASA_HD int sequence_of(int x) const {
    int lo = 0, hi = B;  // Hkv * before(lo) <= x < Hkv * before(hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before(mid) * Hkv <= x) lo = mid;
      else hi = mid;
    }
    return lo;
  }

  // (32-bit arithmetic and no wide divisions: every CTA does this before its first copy)
  FASA_HD int cost_before(int b) const { return Hkv * (before(b) + PAGED_UNIT_COST * b); }
  FASA_HD int cost() const { return cost_before(B); }
  // Its cuts into parts, at most `grid`.
  FASA_HD PagedCuts cuts(int grid) const {
    const int all = cost(), most = (all + PAGED_PART_COST - 1) / PAGED_PART_COST;
    return PagedCuts(all, most < grid ? most : grid);
  }
  // Where part c begins on the line (0 <= c <= n; a part may be empty): the first
  // group that lies at that cost or behind it.
  FASA_HD int part_begin(const PagedCuts& cuts, int c) const {
    const int y = cuts.begin(c);
    if (c >= cuts.n) return total();
    int lo = 0, hi = B;  // cost_before(lo) <= y < cost_before(hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cost_before(mid) <= y) lo = mid;
      else hi = mid;
    }
    const int g = groups(lo), rem = y - cost_before(lo);
    const int h = rem / (g + PAGED_UNIT_COST), off = rem - h * (g + PAGED_UNIT_COST);
    return before(lo) * Hkv + h * g + (off > PAGED_UNIT_COST ? off - PAGED_UNIT_COST : 0);
  }
  // The part that holds group g of unit (b, h).
  FASA_HD int part_of(const PagedCuts& cuts, int b, int h, int g) const {
    const int y = cost_before(b) + h * (groups(b) + PAGED_UNIT_COST) + PAGED_UNIT_COST + g;
    int c = (int)((float)y * cuts.part);  // at most one off
    c = c < cuts.n ? c : cuts.n - 1;
    if (cuts.begin(c) > y) --c;
    else if (c + 1 < cuts.n && cuts.begin(c + 1) <= y) ++c;
    return c;
  }
};

// Walks the units that [x, end) of the line touches.
struct PagedSegments {
  PagedLine line;
  int end;
  int x, b, h;  // where the next segment begins
  int unit_begin, unit_end;

  FASA_HD void start(const PagedLine& l, int x_, int end_) {
    line = l;
    x = x_;
    end = end_;
    b = h = 0;
    if (x < end) {
      b = line.sequence_of(x);
      h = (x - line.before(b) * line.Hkv) / line.groups(b);
    }
  }
  // The segment at x: its unit (b, h) and where the unit lies; false at the end.
  FASA_HD bool at() {
    if (x >= end) return false;
    while (line.groups(b) == 0) ++b;
    const int n = line.groups(b);
    unit_begin = line.before(b) * line.Hkv + h * n;
    unit_end = unit_begin + n;
    return true;
  }
  FASA_HD int unit() const { return b * line.Hkv + h; }
  FASA_HD int seg_end() const { return unit_end < end ? unit_end : end; }
  FASA_HD int first_part(const PagedCuts& cuts) const { return line.part_of(cuts, b, h, 0); }
  FASA_HD int last_part(const PagedCuts& cuts) const {
    return line.part_of(cuts, b, h, unit_end - unit_begin - 1);
  }
  FASA_HD void next() {
    x = seg_end();
    if (x == unit_end && ++h == line.Hkv) {
      h = 0;
      ++b;
    }
  }
};

}  // namespace fasa
