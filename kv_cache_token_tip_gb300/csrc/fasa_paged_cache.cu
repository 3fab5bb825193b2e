// Writing and cutting the paged cache: the append of new tokens and the
// eviction by accumulated attention weight.
#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>

#include "fasa_cluster.cuh"
#include "fasa_internal.h"
#include "fasa_paged.h"
#include "fasa_ptx.cuh"

namespace fasa {
namespace {

// ------------------------------------------------------------------- append
// A warp takes a token and some of its heads' rows, 16 bytes of a row to a lane,
// so that a lane turns the same pairs of every head: the warp computes a token's
// cosines and sines once.  The rows are on their way meanwhile.  Bound by the bytes for a
// prompt (16.5K tokens of 8 heads, 129 MB: 23.9 us, 80% of the copy rate), by the chain
// of loads (table, length, page) for a token a sequence (32 sequences: 1.9 us).
constexpr int AP_NT = 128;
constexpr int AP_U = 2;              // rows of K and of V a lane has on the way
// From this many tokens a warp takes all heads of one: 16.5K tokens 23.8 us against
// 34.0 with two heads a warp; 32 tokens 2.6 us against 2.0.
constexpr int AP_MANY = 2048;

// Sequence of new token x, and which of its tokens it is; false for padding (used:
// cu_new[B]) and where the table does not ascend about x (reported).  A whole warp.
__device__ __forceinline__ bool token_of(const PagedAppendParams& p, int x, int used, int& b, int& j) {
  const int lane = threadIdx.x & 31;
  if (x >= used) return false;  // padding
  int lo = 0, hi = p.B;  // cu_new[lo] <= x < cu_new[hi]: 32 places at a time
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    lo += __popc(__ballot_sync(0xffffffffu, at < hi && p.cu_new[min(at, p.B)] <= x)) * step;
    hi = min(hi, lo + step);
  }
  const int first = p.cu_new[lo], next = p.cu_new[lo + 1];
  b = lo;
  j = x - first;
  if (first < 0 || first > x || next <= x || next > p.n_tokens) {
    if (lane == 0) atomicOr(p.status, 1);
    return false;
  }
  return true;
}

// Four or two pairs of a row, turned.
template <typename T, int NP>
__device__ __forceinline__ uint4 turn_row(const uint4& w, const float2 (&cs)[NP]) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    float x0, x1;
    if constexpr (sizeof(T) == 2) {
      x0 = bf16_lo(in[i]);
      x1 = bf16_hi(in[i]);
    } else {
      x0 = __uint_as_float(in[2 * i]);
      x1 = __uint_as_float(in[2 * i + 1]);
    }
    const float y0 = x0 * cs[i].x - x1 * cs[i].y, y1 = x0 * cs[i].y + x1 * cs[i].x;
    if constexpr (sizeof(T) == 2) {
      out[i] = pack_bf16(y0, y1);
    } else {
      out[2 * i] = __float_as_uint(y0);
      out[2 * i + 1] = __float_as_uint(y1);
    }
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// heads: of a warp, whole steps of the rows its lanes cover.  TABLE: with a table of rows,
// or a token a sequence (which then pays nothing for the table: 32 sequences 1.9 us, 2.1
// with one kernel for both).
template <typename T, int D, bool TABLE>
__global__ void __launch_bounds__(AP_NT) paged_append_kernel(const __grid_constant__ PagedAppendParams p, int heads) {
  constexpr int LPR = D * (int)sizeof(T) / 16, RPW = 32 / LPR;  // lanes of a row, rows of a warp
  constexpr int EPL = 16 / (int)sizeof(T), NP = EPL / 2;        // elements and pairs of a lane
  __shared__ unsigned long long turns[D / 2];
  __shared__ __align__(16) float2 angles[AP_NT / 32][D / 2];  // cos and sin of a warp's token
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // (lanes reading different parameter words take turns: some lanes of each warp)
  constexpr int TW = D / 2 / (AP_NT / 32);
  if (lane < TW) turns[warp * TW + lane] = p.rope_turns[warp * TW + lane];
  __syncthreads();
  paged_go();
  paged_wait();
  // A table of rows is checked whole, by a block of its own: the tokens look at their
  // own sequence's range alone, and padding at none.  (8 sequences with a token each
  // 2.45 us, 1500 of two 3.42, 8 of 700 7.29; without the check 2.36, 3.27, 7.11; checked
  // by the last block behind its tokens 2.55, 5.33, 7.20.)
  constexpr int own = TABLE;
  if (TABLE && blockIdx.x == 0) {
    int bad = 0;
#pragma unroll 4
    for (int i = threadIdx.x; i <= p.B; i += AP_NT) {
      const int x = p.cu_new[i], low = p.cu_new[max(i - 1, 0)];
      bad |= (x < low) | (x > p.n_tokens) | (i == 0 && x != 0);
    }
    if (bad) atomicOr(p.status, 1);
    return;
  }
  const int chunks = (p.Hkv + heads - 1) / heads, at = lane % LPR, sub = lane / LPR;
  const long long items = (long long)p.n_tokens * chunks, warps = (long long)(gridDim.x - own) * (AP_NT / 32);
  const int used = TABLE ? p.cu_new[p.B] : p.n_tokens;
  for (long long w = (long long)(blockIdx.x - own) * (AP_NT / 32) + warp; w < items; w += warps) {
    const int x = (int)(w / chunks), h0 = (int)(w - (long long)x * chunks) * heads, h1 = min(p.Hkv, h0 + heads);
    // the rows first: they need only x, the rest is a chain of loads
    uint4 k[AP_U], v[AP_U];
    auto load = [&](int hb) {
#pragma unroll
      for (int i = 0; i < AP_U; ++i) {
        const int h = hb + i * RPW + sub;
        const size_t from = ((size_t)x * p.Hkv + h) * D + at * EPL;
        if (h < h1) {
          k[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.k_new) + from);
          v[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.v_new) + from);
        }
      }
    };
    load(h0);
    int b, j;
    if constexpr (TABLE) {
      if (!token_of(p, x, used, b, j)) continue;
    } else {
      b = x;
      j = 0;
    }
    const int len = p.seq_lens[b], m = p.pos[b] + j;
    const long long slot = (long long)len + j;
    if (len < 0 || slot >= p.T_cap) {
      if (lane == 0) atomicOr(p.status, 1);
      continue;
    }
    const int page = p.page_table[(size_t)b * p.max_pages + (slot >> p.log2_page)];
    if (page < 0 || page >= p.n_pages) {
      if (lane == 0) atomicOr(p.status, 1);
      continue;
    }
    __syncwarp();  // (the last token's are read)
#pragma unroll 1
    for (int f = lane; f < D / 2; f += 32) angles[warp][f] = rope_cos_sin(turns[f], m);
    __syncwarp();
    float2 cs[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) cs[i] = angles[warp][at * NP + i];
    for (int hb = h0; hb < h1; hb += RPW * AP_U) {
      if (hb > h0) load(hb);
#pragma unroll
      for (int i = 0; i < AP_U; ++i) {
        const int h = hb + i * RPW + sub;
        if (h < h1) {
          const size_t to = (size_t)paged_row(page, p.n_pages, p.Hkv, h, p.log2_page, (int)slot) * D + at * EPL;
          *reinterpret_cast<uint4*>(static_cast<T*>(p.k_pages) + to) = turn_row<T, NP>(k[i], cs);
          *reinterpret_cast<uint4*>(static_cast<T*>(p.v_pages) + to) = v[i];
          if (at == 0) {
            const size_t stat = ((size_t)b * p.Hkv + h) * p.T_cap + slot;
            if (p.weight) p.weight[stat] = 0.f;
            if (p.token_pos) p.token_pos[stat] = m;
          }
        }
      }
    }
  }
}

// -------------------------------------------------------------------- evict
// One cluster per (sequence, KV head), each CTA a contiguous share of its slots
// with their keys in shared memory.
//   1. Keys: held tokens above every weight, NaN below every number, else the
//      weight's order-preserving bits.
//   2. Up to EV_FEW tokens too many, as in a decode loop: the last of the order is
//      found and struck out, one after the other, and the few moves that this leaves
//      are made at once.
//      More: the cluster's least and largest key and its count of held tokens, then
//      the keep-th largest key: a histogram of 2048 bins over the range of the
//      keys, summed over the cluster slice by slice, gives the bin it falls in.
//      A bin that is kept whole ends it; a bin of few keys is sent to every CTA
//      and ranked there by (key, slot); else the bin becomes the range.  A single
//      key held by many slots (ties) goes by slot order.
//   3. Holes and movers, counted over the cluster and listed in slot order; the i-th
//      mover's row goes to the i-th hole by CTA i % C, which takes its part of the
//      list into shared memory first.
// Bound by the latency of these steps (cluster barriers, dependent loads): of the
// 21.4 us that 8 heads of 32K tokens cut to 4096 take, keys and range are 2.6, the
// choice 6.1, holes and movers counted and listed 3.9, and the copies of 28.7 MB there
// and back 4 to 8.7 from CTA to CTA, the last of which ends it; 256 heads of 1900 to 2080
// tokens cut to 2048 take 10.0 us.
constexpr int EV_NW = 16;            // most warps of a CTA
constexpr int EV_BINS = 2048;
constexpr int EV_CAND = 512;         // keys of a bin that are ranked one by one
// Tokens that are struck out one by one.  One, four, eight over the bound, 8 heads of
// 4096: 4.1, 5.9, 8.2 us against 8.9, 9.2, 8.9 with the histogram; 64 heads of 4096: 4.5,
// 6.7, 9.6 against 10.4, 10.8, 11.0; sixteen over: 15.5 and 17.8 against 9.7 and 11.4.
constexpr int EV_FEW = 8;
constexpr int EV_LIST = 1536;        // moves in a CTA's shared memory, where its histogram was
constexpr int EV_MAX_SHARE = 16384;  // slots of a CTA: 64 KB of keys
constexpr int EV_SHORT_SHARE = 2048;  // (8 heads of 32K: 21.3 us, 26.9 with shares of 4096)
constexpr int EV_C_MAX = 16;
// More CTAs to an SM than this, and they have 256 threads, not 512, so that twice as
// many units are under way: 384, 512, 2048 units one token over 2048: 6.0, 6.0, 25.5 us
// against 7.8, 8.7, 35.7; 512 of 4096 halved, which is copies: 118 against 110; 256
// units have no SM to share: 5.5 against 4.8.
constexpr int EV_NARROW = 2;

struct EvictShared {
  union {
    struct {
      int hist[EV_BINS];
      int slice[EV_BINS];        // this CTA's slice of the cluster's histogram
      int partial[EV_BINS / 2];  // its sums over some of the CTAs
      unsigned long long cand[EV_CAND];  // key, then ~slot: a larger entry comes first
    };
    PagedMove moves[EV_LIST];  // once the choice is made: those that this CTA makes
  };
  int4 facts[EV_C_MAX];      // every CTA's least and largest key and held tokens
  uint2 last_of_warp[2][EV_NW], last[2][EV_C_MAX];  // the last in the order: key, ~slot
  int slice_sum[EV_C_MAX];
  int tie_sum[EV_C_MAX];
  int2 sums[EV_C_MAX];       // every CTA's holes and movers
  int scan[EV_NW];
  int4 red[EV_NW];
  int bin, above, cnt, n_cand;
};

// What the selection orders by: held tokens above every weight, NaN below (and 0 is
// for what is struck out).
__device__ __forceinline__ unsigned evict_key(float w, int tp, int sinks, long long recent_after) {
  if (tp < sinks || (long long)tp > recent_after) return 0xffffffffu;
  return w != w ? 1u : score_key(w);
}

// The warp's least pair, by x, then y.
__device__ __forceinline__ uint2 warp_least(uint2 v) {
  const unsigned x = __reduce_min_sync(0xffffffffu, v.x);
  return make_uint2(x, __reduce_min_sync(0xffffffffu, v.x == x ? v.y : 0xffffffffu));
}

// Exclusive prefix sum over the block (thread order) and the total.
template <int NT>
__device__ int block_scan(int x, int* scan, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  const int v = lane < NT / 32 ? scan[lane] : 0;
  const int below = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
  total = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  return below + incl - x;
}

template <int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) paged_evict_kernel(const __grid_constant__ PagedEvictParams p) {
  extern __shared__ __align__(16) unsigned keys[];
  __shared__ EvictShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)cluster_size(), rank = (int)cluster_rank();
  const int u = blockIdx.x / C, b = u / p.Hkv, h = u - b * p.Hkv;
  auto csync = [&]() {
    if (C > 1) cluster_sync();
    else __syncthreads();
  };
  for (int i = tid; i < EV_BINS; i += NT) sh.hist[i] = 0;
  if (tid == 0) sh.n_cand = 0;
  paged_go();
  paged_wait();
  int len = p.seq_lens[b];
  if (len < 0 || len > p.T_cap) {
    if (tid == 0) atomicOr(p.status, 1);
    len = min(max(len, 0), p.T_cap);
  }
  const int keep = p.keep, left = min(len, keep);
  if (h == 0 && rank == 0 && tid == 0) p.new_lens[b] = left;
  const size_t base = (size_t)u * p.T_cap;
  const float* w = p.weight + base;
  const int* tp = p.token_pos + base;
  float* wo = p.weight_out + base;
  int* to = p.token_pos_out + base;
  const bool apart = wo != w;
  if (len <= keep && !apart) return;
  if (C > 1 && len > keep) cluster_arrive_relaxed();  // (the cluster's CTAs have started before one writes to another)
  // this CTA's slots: [first, first + n), whole groups of four but the last
  const int share = ((len + C - 1) / C + 3) & ~3;
  const int first = min(len, rank * share), n = min(len - first, share);
  // 1. keys (T_cap is whole groups: a vector may pass len, its extra keys are unused)
  const long long after = (long long)p.pos[b] - p.recent;
  unsigned mn = 0xffffffffu, mx = 0u;
  int held = 0;
  for (int i = 4 * tid; i < n; i += 4 * NT) {
    const int t = first + i;
    const float4 wv = *reinterpret_cast<const float4*>(w + t);
    const int4 tv = *reinterpret_cast<const int4*>(tp + t);
    if (apart) {  // into other buffers: the holes among these are written over below
      if (t + 4 <= left) {
        *reinterpret_cast<float4*>(wo + t) = wv;
        *reinterpret_cast<int4*>(to + t) = tv;
      } else {
        const float we[4] = {wv.x, wv.y, wv.z, wv.w};
        const int te[4] = {tv.x, tv.y, tv.z, tv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (t + e < left) {
            wo[t + e] = we[e];
            to[t + e] = te[e];
          }
      }
    }
    const unsigned k[4] = {evict_key(wv.x, tv.x, p.sinks, after), evict_key(wv.y, tv.y, p.sinks, after),
                           evict_key(wv.z, tv.z, p.sinks, after), evict_key(wv.w, tv.w, p.sinks, after)};
    *reinterpret_cast<uint4*>(keys + i) = make_uint4(k[0], k[1], k[2], k[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n) {
        if (k[e] == 0xffffffffu) {
          ++held;
        } else {
          mn = min(mn, k[e]);
          mx = max(mx, k[e]);
        }
      }
  }
  if (len <= keep) return;
  // 2.
  if (len - keep <= EV_FEW) {
    if (C > 1) cluster_wait();
    __syncthreads();  // (a thread's keys for this are not those it wrote)
    auto last_of_mine = [&]() {
      uint2 v = make_uint2(0xffffffffu, 0xffffffffu);
      for (int i = tid; i < n; i += NT) {
        const unsigned k = keys[i], s = ~(unsigned)(first + i);
        if (k != 0u && (k < v.x || (k == v.x && s < v.y))) v = make_uint2(k, s);
      }
      return v;
    };
    uint2 mine = last_of_mine();
    const int few = len - keep;
    int gone = 0x7fffffff;  // lane i's: the slot struck out i-th
#pragma unroll 1
    for (int i = 0; i < few; ++i) {
      const int side = i & 1;
      uint2 v = warp_least(mine);
      if (lane == 0) sh.last_of_warp[side][warp] = v;
      __syncthreads();
      v = warp_least(sh.last_of_warp[side][lane & (NT / 32 - 1)]);
      if (C > 1) {
        if (tid < C) dsmem_st_v2u32(dsmem_map(smem_u32(&sh.last[side][rank]), tid), v.x, v.y);
        cluster_sync();
        v = warp_least(sh.last[side][lane & (C - 1)]);
      }
      if (lane == i) gone = (int)~v.y;
      if (v.x == mine.x && v.y == mine.y) {
        keys[(int)~v.y - first] = 0u;
        mine = last_of_mine();
      }
    }
    // every warp knows them all: the first CTA's move the few rows, 16 bytes a thread,
    // holes and movers in slot order
    if (rank != 0) return;
    const int log2_n16 = 31 - __clz(p.row_bytes / 16), log2_move = log2_n16 + 1;
    const int part = tid & ((1 << log2_move) - 1);
    char* pool = static_cast<char*>((part >> log2_n16) ? p.v_pages : p.k_pages) + (part & ((1 << log2_n16) - 1)) * 16;
    const int* table = p.page_table + (size_t)b * p.max_pages;
    int before = 0;
    for (int i = 0; i < few; ++i) before += __shfl_sync(0xffffffffu, gone, i) < gone;
    const unsigned all_kept = ((1u << few) - 1u) &
                              ~__reduce_or_sync(0xffffffffu, lane < few && gone >= keep ? 1u << (gone - keep) : 0u);
    for (int m0 = 0; m0 < few; m0 += NT >> log2_move) {
      const int move = m0 + (tid >> log2_move);
      int hole = keep;
      for (int i = 0; i < few; ++i) {
        const int at = __shfl_sync(0xffffffffu, before, i), x = __shfl_sync(0xffffffffu, gone, i);
        hole = at == move ? x : hole;
      }
      if (hole >= keep) continue;
      unsigned kept = all_kept;
      for (int i = 0; i < move; ++i) kept &= kept - 1u;
      const int mover = keep + __ffs(kept) - 1;
      const long long dst = paged_row(table[hole >> p.log2_page], p.n_pages, p.Hkv, h, p.log2_page, hole);
      const long long src = paged_row(table[mover >> p.log2_page], p.n_pages, p.Hkv, h, p.log2_page, mover);
      if (dst >= 0 && src >= 0)
        *reinterpret_cast<uint4*>(pool + dst * p.row_bytes) = *reinterpret_cast<const uint4*>(pool + src * p.row_bytes);
      else if (part == 0)
        atomicOr(p.status, 1);
      if (part == 0) {
        wo[hole] = w[mover];
        to[hole] = tp[mover];
      }
    }
    return;
  }
  mn = __reduce_min_sync(0xffffffffu, mn);
  mx = __reduce_max_sync(0xffffffffu, mx);
  held = __reduce_add_sync(0xffffffffu, held);
  if (lane == 0) sh.red[warp] = make_int4((int)mn, (int)mx, held, 0);
  __syncthreads();
  if (C > 1) cluster_wait();
  if (warp == 0) {  // to every CTA
    const int4 r = lane < NT / 32 ? sh.red[lane] : make_int4(-1, 0, 0, 0);
    mn = __reduce_min_sync(0xffffffffu, (unsigned)r.x);
    mx = __reduce_max_sync(0xffffffffu, (unsigned)r.y);
    held = __reduce_add_sync(0xffffffffu, r.z);
    if (lane < C)
      dsmem_st_v4u32(dsmem_map(smem_u32(&sh.facts[rank]), lane), make_uint4(mn, mx, (unsigned)held, 0u));
  }
  csync();
  // kept: keys from `floor` on, and of tie_key the first `need` slots
  unsigned tie_key = 0xffffffffu, lo = 0xffffffffu, hi = 0u;
  int need = 0;
  held = 0;
  for (int r = 0; r < C; ++r) {
    lo = min(lo, (unsigned)sh.facts[r].x);
    hi = max(hi, (unsigned)sh.facts[r].y);
    held += sh.facts[r].z;
  }
  int kr = keep - held;
  unsigned long long floor = kr == 0 ? 0xffffffffull : 1ull << 32;
  if (kr < 0) need = keep;  // more held tokens than room
  const int SL = EV_BINS / C;
  for (bool again = false; kr > 0; again = true) {
    const int shift = max(0, 32 - __clz(hi - lo) - 11);
    if (again) {  // (zeros before the first)
      for (int i = tid; i < EV_BINS; i += NT) sh.hist[i] = 0;
      __syncthreads();
    }
    for (int i = tid; i < n; i += NT) {
      const unsigned k = keys[i];
      if (k >= lo && k <= hi) atomicAdd(&sh.hist[(k - lo) >> shift], 1);
    }
    csync();
    // this CTA's slice of the bins, over the cluster: a thread takes a bin of some
    // of the CTAs
    int sum = 0;
    if (C == 1) {
      for (int i = tid; i < SL; i += NT) sum += sh.slice[i] = sh.hist[i];
    } else {
      const int np = max(1, NT / SL), part = tid / SL;  // (SL 1024: two bins a thread)
      for (int i = tid - part * SL; i < SL; i += NT) {
        const uint32_t at = smem_u32(&sh.hist[rank * SL + i]);
        int v = 0;
#pragma unroll 4
        for (int r = part; r < C; r += np) v += (int)dsmem_ld_u32(dsmem_map(at, r));
        sh.partial[part * SL + i] = v;
      }
      __syncthreads();
      for (int i = tid; i < SL; i += NT) {
        int v = 0;
        for (int q = 0; q < np; ++q) v += sh.partial[q * SL + i];
        sh.slice[i] = v;
        sum += v;
      }
    }
    int total;
    block_scan<NT>(sum, sh.scan, total);
    if (tid < C) dsmem_st_u32(dsmem_map(smem_u32(&sh.slice_sum[rank]), tid), (uint32_t)total);
    csync();
    // the slice, then the bin of it, that holds the kr-th key from the top
    int above = 0, owner = C - 1;
    while (owner > 0 && above + sh.slice_sum[owner] < kr) above += sh.slice_sum[owner--];
    const int per = max(1, SL / NT);
    int c[EV_BINS / NT], mine = 0;
#pragma unroll
    for (int j = 0; j < EV_BINS / NT; ++j) {
      const int at = SL - 1 - (tid * per + j);
      c[j] = j < per && at >= 0 ? (int)dsmem_ld_u32(dsmem_map(smem_u32(&sh.slice[max(at, 0)]), owner)) : 0;
      mine += c[j];
    }
    above += block_scan<NT>(mine, sh.scan, total);
#pragma unroll
    for (int j = 0; j < EV_BINS / NT; ++j) {
      if (above < kr && kr <= above + c[j]) {
        sh.bin = owner * SL + SL - 1 - (tid * per + j);
        sh.above = above;
        sh.cnt = c[j];
      }
      above += c[j];
    }
    __syncthreads();
    const int bin = sh.bin, cnt = sh.cnt;
    kr -= sh.above;
    const unsigned b0 = lo + ((unsigned)bin << shift);
    const unsigned b1 = b0 + min(hi - b0, (1u << shift) - 1u);  // its last key
    if (cnt == kr) {  // kept whole
      floor = b0;
      break;
    }
    if (cnt <= EV_CAND) {
      // every CTA gets all keys of the bin, CTA after CTA, and marks its own as
      // kept (largest key) or not (least)
      const int before = (int)__reduce_add_sync(
          0xffffffffu, lane < rank ? dsmem_ld_u32(dsmem_map(smem_u32(&sh.hist[bin]), lane)) : 0u);
      for (int i = tid; i < n; i += NT) {
        const unsigned k = keys[i];
        if (k >= b0 && k <= b1) {
          const int at = before + atomicAdd(&sh.n_cand, 1);
          for (int r = 0; r < C; ++r)
            dsmem_st_v2u32(dsmem_map(smem_u32(&sh.cand[at]), r), ~(unsigned)(first + i), k);
        }
      }
      csync();
      for (int i = tid; i < cnt; i += NT) {
        const unsigned long long e = sh.cand[i];
        const int slot = (int)~(unsigned)e;
        if (slot < first || slot >= first + n) continue;
        int above_me = 0;
#pragma unroll 8
        for (int q = 0; q < cnt; ++q) above_me += sh.cand[q] > e;
        keys[slot - first] = above_me < kr ? 0xffffffffu : 0u;
      }
      floor = max(b0, 1u);
      break;
    }
    if (shift == 0) {  // one key in many slots
      tie_key = b0;
      floor = (unsigned long long)b0 + 1ull;
      need = kr;
      break;
    }
    lo = b0;
    hi = b1;
  }
  __syncthreads();
  // 3. holes and movers: a thread has a run of slots
  const int run = ((n + NT - 1) / NT + 3) & ~3;
  const int i0 = min(n, tid * run), i1 = min(n, i0 + run);
  const int* table = p.page_table + (size_t)b * p.max_pages;
  int page_at = -1, page = -1;  // the table's entry at page_at, for the run's first slot ahead
  if (i0 < i1) {
    page_at = (first + i0) >> p.log2_page;
    page = table[page_at];
  }
  int ties = 0, total;
  if (need) {
    for (int i = i0; i < i1; ++i) ties += keys[i] == tie_key;
    const int mine = ties;
    ties = block_scan<NT>(mine, sh.scan, total);
    if (tid < C) dsmem_st_u32(dsmem_map(smem_u32(&sh.tie_sum[rank]), tid), (uint32_t)total);
    csync();
    for (int r = 0; r < rank; ++r) ties += sh.tie_sum[r];
  }
  auto walk = [&](auto&& visit) {
    int tie = ties;
    for (int i = i0; i < i1; ++i) {
      const unsigned k = keys[i];
      bool kept = (unsigned long long)k >= floor;
      if (need && k == tie_key) kept = kept || tie++ < need;
      const int t = first + i;
      visit(t, t < keep && !kept, t >= keep && kept);
    }
  };
  int holes = 0, movers = 0;
  walk([&](int, bool hole, bool mover) {
    holes += hole;
    movers += mover;
  });
  // (both counts of a CTA are below 2^15)
  const int packed = block_scan<NT>(holes | movers << 16, sh.scan, total);
  if (tid < C)
    dsmem_st_v2u32(dsmem_map(smem_u32(&sh.sums[rank]), tid), (uint32_t)(total & 0xffff), (uint32_t)(total >> 16));
  csync();
  int hole_at = packed & 0xffff, mover_at = packed >> 16, moves_n = 0;
  for (int r = 0; r < C; ++r) {
    if (r < rank) {
      hole_at += sh.sums[r].x;
      mover_at += sh.sums[r].y;
    }
    moves_n += sh.sums[r].x;
  }
  PagedMove* listed = p.moves + (size_t)u * p.move_cap;
  if (holes + movers) {
    walk([&](int t, bool hole, bool mover) {
      if (!hole && !mover) return;
      if (t >> p.log2_page != page_at) {
        page_at = t >> p.log2_page;
        page = table[page_at];
      }
      const int row = (int)paged_row(page, p.n_pages, p.Hkv, h, p.log2_page, t);
      if (row < 0) atomicOr(p.status, 1);
      const int at = hole ? hole_at++ : mover_at++;
      (hole ? listed[at].hole : listed[at].mover) = make_int2(row, t);
    });
  }
  csync();  // (and no CTA reads another's shared memory behind it)
  // 4. the copies: 16 bytes a thread, several of them on the way (32K to 4096: 22.1 us
  // with four, 21.4 with five or seven, which are slower where few rows move)
  constexpr int U = 5;
  const int log2_n16 = 31 - __clz(p.row_bytes / 16), log2_move = log2_n16 + 1;
  const int part = tid & ((1 << log2_move) - 1);  // the same for all of a thread's items
  char* pool = static_cast<char*>((part >> log2_n16) ? p.v_pages : p.k_pages) + (part & ((1 << log2_n16) - 1)) * 16;
  const int log2_C = 31 - __clz(C), own = (moves_n + C - 1 - rank) >> log2_C;  // move i is CTA i % C's
  for (int m0 = 0; m0 < own; m0 += EV_LIST) {
    const int n_moves = min(own - m0, EV_LIST);
    if (m0) __syncthreads();  // the last ones are read
    for (int i = tid; i < n_moves; i += NT)
      *reinterpret_cast<int4*>(&sh.moves[i]) =
          ld_cg(reinterpret_cast<const int4*>(listed + ((size_t)(m0 + i) << log2_C) + rank));
    __syncthreads();
    const int items = n_moves << log2_move;
    for (int q0 = tid; q0 < items; q0 += U * NT) {
      uint4 v[U];
      int into[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int q = q0 + j * NT;
        const PagedMove m = q < items ? sh.moves[q >> log2_move] : PagedMove{make_int2(-1, 0), make_int2(-1, 0)};
        into[j] = m.mover.x >= 0 ? m.hole.x : -1;
        if (into[j] >= 0) v[j] = ld_cg(reinterpret_cast<const uint4*>(pool + (long long)m.mover.x * p.row_bytes));
      }
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (into[j] >= 0) *reinterpret_cast<uint4*>(pool + (long long)into[j] * p.row_bytes) = v[j];
    }
    for (int i = tid; i < n_moves; i += NT) {
      const PagedMove m = sh.moves[i];
      wo[m.hole.y] = w[m.mover.y];
      to[m.hole.y] = tp[m.mover.y];
    }
  }
}

}  // namespace

namespace {

template <typename T, int D>
cudaError_t launch_append(const PagedAppendParams& p, int sms, cudaStream_t s) {
  // few tokens: as many warps as rows allow; many: a token's cosines once
  constexpr int RPW = 32 / (D * (int)sizeof(T) / 16);
  const int heads = p.n_tokens < AP_MANY ? RPW : (p.Hkv + RPW - 1) / RPW * RPW;
  const long long items = (long long)p.n_tokens * ((p.Hkv + heads - 1) / heads);
  const long long blocks = (items + AP_NT / 32 - 1) / (AP_NT / 32) + (p.cu_new != nullptr);  // (one looks at the table)
  return paged_behind(p.cu_new ? paged_append_kernel<T, D, true> : paged_append_kernel<T, D, false>,
                      (unsigned)(blocks < 16ll * sms ? blocks : 16ll * sms), AP_NT, 0, 0, s, p, heads);
}

template <int NT>
cudaError_t launch_evict(const PagedEvictParams& p, int C, int smem, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (!(done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(paged_evict_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, EV_MAX_SHARE * 4);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(paged_evict_kernel<NT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_release);
  }
  return paged_behind(paged_evict_kernel<NT>, (unsigned)(p.B * p.Hkv * C), NT, (size_t)smem, (unsigned)C, s, p);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, int head_dim, bool bf16, int sms, cudaStream_t s) {
  using B16 = __nv_bfloat16;
  if (bf16) return head_dim == 128 ? launch_append<B16, 128>(p, sms, s) : launch_append<B16, 64>(p, sms, s);
  return head_dim == 128 ? launch_append<float, 128>(p, sms, s) : launch_append<float, 64>(p, sms, s);
}

cudaError_t launch_paged_evict(const PagedEvictParams& p, int sms, cudaStream_t s) {
  const int units = p.B * p.Hkv;
  // CTAs to a unit: a share must fit, and while the units alone leave SMs idle a
  // share of 2048 slots is as short as its steps' latency is worth
  int C = 1;
  while (C < EV_C_MAX &&
         (p.T_cap > C * EV_MAX_SHARE || (p.T_cap > C * EV_SHORT_SHARE && units * C < sms)))
    C *= 2;
  const int smem = min(((p.T_cap + C - 1) / C + 3) & ~3, EV_MAX_SHARE) * 4;
  const bool narrow = (long long)units * C > EV_NARROW * sms;
  return narrow ? launch_evict<256>(p, C, smem, s) : launch_evict<512>(p, C, smem, s);
}

}  // namespace fasa
