// Index arithmetic of the attention of chunks, for the kernels and (as plain C++)
// for the host tests: the split of the work over the CTAs.
//
// Sequence b has n new tokens, the last n of its len slots, taken T at a time: tile
// i of them holds T tokens with the G heads of a KV head as rows.  Unit (b, h, i) is
// that tile of KV head h; it reads the slots that its last token sees, in tiles of
// KT.  All units in order form one line, cut into parts of equal cost, one to a CTA:
// a unit costs its start and its end, `unit`, and a count of slots,
// a + (i + 1) T, a = max(len - n, 0), no less than it reads, whose sum over i is a
// formula, so that a part finds its place without a list of units.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define FASA_CHUNK_HD __host__ __device__ __forceinline__
#else
#define FASA_CHUNK_HD inline
#endif

namespace fasa {

constexpr int CHUNK_MAX_SMS = 160;    // the workspace has room for their parts

// Tokens of a unit (their rows: times the heads of their group), slots of a tile, and what a
// unit costs beside its tiles, in slots.  bf16: a start and an end take as long as 290 slots in a
// traced build; more than that was picked by times, and calls of few rows pay for it.  With 128,
// 256, 384, 512 and 768: eight prompts of 37 to 4096 tokens 377, 359, 322, 311 and 323 us, eight of
// 1000 110, 108, 109, 106 and 110, a server's step 298, 284, 273, 269 and 268; drafted tokens 111,
// 110, 111, 113 and 114, 64 tokens behind 4000 26.5, 28.4, 28.0, 28.1 and 27.7, 8 behind 1000 13.6,
// 13.7, 14.2, 14.7 and 14.2.  fp32, with 16, 48 and 128: two prompts 238, 230 and 236, 65 tokens
// behind 959 34.5, 34.5 and 35.0.
struct ChunkShape {
  int tokens, tile, unit;
};
constexpr int CHUNK_TILE_BF16 = 128, CHUNK_UNIT_BF16 = 512, CHUNK_TILE_F32 = 64, CHUNK_UNIT_F32 = 48;
inline ChunkShape chunk_shape(bool bf16, int G) {
  return bf16 ? ChunkShape{2 * (128 / G), CHUNK_TILE_BF16, CHUNK_UNIT_BF16} : ChunkShape{128 / G, CHUNK_TILE_F32, CHUNK_UNIT_F32};
}

// A sequence's new tokens, where they begin among the call's rows, and its slots.
struct ChunkSeq {
  int first, n, len;
};

struct ChunkLine {
  const long long* before;  // [B + 1]: cost of one head of the sequences before b
  const int* cu_new;        // null: a token a sequence
  const int* seq_lens;
  int n_tokens, T_cap, B, Hkv, T, KT, unit;

  // Sequence b as far as it fits: no token of a range that is not within the call's rows.
  FASA_CHUNK_HD ChunkSeq sequence(int b, bool* bad) const {
    ChunkSeq q;
    const int len = seq_lens[b];
    q.len = len < 0 ? 0 : len > T_cap ? T_cap : len;
    *bad = *bad || q.len != len;
    q.first = b;
    q.n = 1;
    if (cu_new) {
      const int end = cu_new[b + 1];
      q.first = cu_new[b];
      const bool ok = 0 <= q.first && q.first <= end && end <= n_tokens;
      q.n = ok ? end - q.first : 0;
      *bad = *bad || !ok || (b == 0 && q.first != 0);
    }
    return q;
  }
  FASA_CHUNK_HD static int tiles_of(int n, int T) { return (n + T - 1) / T; }
  // Cost of the first i units of a head of a sequence.
  FASA_CHUNK_HD long long cost_of(int n, int len, int i) const {
    const long long a = len > n ? len - n : 0;
    return (long long)i * (unit + a) + (long long)T * i * (i + 1) / 2;
  }
  FASA_CHUNK_HD long long cost_of(int n, int len) const { return cost_of(n, len, tiles_of(n, T)); }

  FASA_CHUNK_HD long long total() const { return before[B] * Hkv; }
  FASA_CHUNK_HD int parts(int most) const {
    const long long t = total(), n = (t + KT - 1) / KT;  // (no part is shorter than a tile)
    return n < most ? (int)n : most;
  }
  FASA_CHUNK_HD long long part_begin(int parts, int c) const {
    const long long t = total();
    return c >= parts ? t : t / parts * c + t % parts * c / parts;
  }
};

// A place on the line: a unit, where it begins, and how many of its tiles lie before a
// cut there.
struct ChunkUnit {
  int b, h, i;
  ChunkSeq q;
  long long begin, cost;
  int tiles;  // that its last token sees

  FASA_CHUNK_HD void fill(const ChunkLine& l) {
    const int last = (i + 1) * l.T < q.n ? (i + 1) * l.T : q.n;
    const int see = q.len - q.n + last;  // (all of len at most)
    tiles = see > 0 ? (see + l.KT - 1) / l.KT : 0;
    cost = l.unit + (q.len > q.n ? q.len - q.n : 0) + (long long)(i + 1) * l.T;
  }
  // The unit that holds position y, 0 <= y < total.
  FASA_CHUNK_HD void find(const ChunkLine& l, long long y) {
    int lo = 0, hi = l.B;  // Hkv before(lo) <= y < Hkv before(hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (l.before[mid] * l.Hkv <= y) lo = mid;
      else hi = mid;
    }
    b = lo;
    bool bad = false;
    q = l.sequence(b, &bad);
    const long long head = l.before[b + 1] - l.before[b];
    begin = l.before[b] * l.Hkv;
    y -= begin;
    h = (int)(y / head);
    y -= h * head;
    lo = 0;
    hi = ChunkLine::tiles_of(q.n, l.T);
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (l.cost_of(q.n, q.len, mid) <= y) lo = mid;
      else hi = mid;
    }
    i = lo;
    begin += h * head + l.cost_of(q.n, q.len, i);
    fill(l);
  }
  // The unit behind this one; only where there is one.
  FASA_CHUNK_HD void next(const ChunkLine& l) {
    begin += cost;
    if (++i == ChunkLine::tiles_of(q.n, l.T)) {
      i = 0;
      if (++h == l.Hkv) {
        h = 0;
        do ++b;
        while (l.before[b + 1] == l.before[b]);
        bool bad = false;
        q = l.sequence(b, &bad);
      }
    }
    fill(l);
  }
  // Tiles of the unit that lie before position y: tile 0 at its begin, tile t at
  // unit + KT t behind it.
  FASA_CHUNK_HD int before(const ChunkLine& l, long long y) const {
    if (y <= begin) return 0;
    if (y >= begin + cost) return tiles;
    const long long r = y - begin - l.unit;
    const int t = r > 0 ? (int)((r + l.KT - 1) / l.KT) : 0;
    const int at_least = t > 1 ? t : 1;
    return at_least < tiles ? at_least : tiles;
  }
};

}  // namespace fasa
