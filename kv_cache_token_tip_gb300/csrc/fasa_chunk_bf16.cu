// Attention of chunks in bf16 on the 5th-generation tensor cores.  A block takes a
// part of the line of units (fasa_chunk_index.h): two tiles of up to 128 rows (new
// tokens times the heads of their group), the slots 128 at a time.
//
// Per tile of rows and of slots: S = Q K^T (fp32, tensor memory), P = 2^(scale S - m) by
// a warpgroup, a row to a thread, back to tensor memory in bf16 over S, O += P V.  m
// follows the row's maximum only where it rises by more than 2^8: O is seldom scaled, and
// out = O / sum P is the same.  Roles: a warpgroup for each tile of rows, a warp that
// issues the matrix instructions, one that copies.  While the tensor cores work for one tile
// of rows, the softmax of the other is worked out.
//
// Bound by the tensor cores where units are long: 2048 tokens behind 30720 take 610 to 630 us by
// themselves (tensor pipe 81% busy), and 690 to 740 one after another, where the card's power
// bounds them.  Eight prompts of 37 to 4096 tokens 295 to 305 us (64%): a unit's start and end cost
// 5400 to 5800 clocks beside 2530 a tile (in a traced build).  Drafted tokens of 16 sequences 113
// us, 5.7 TB/s.  What it took, one step after another: instructions issued by one elected lane from
// descriptors worked out ahead (742 -> 684 us for the first case), P handed over by halves and a row
// to a thread (598; half a row to each of two warps 684), results by way of shared memory (eight
// prompts 372 -> 327), what a unit costs (fasa_chunk_index.h).
//
// P is rounded to bf16, an operand's type here: results are off by 2.2e-3 to 2.3e-3 of their norm
// where weights in fp32, and one rounding of the result, give 1.6e-3 to 1.7e-3.  P in two terms
// would bring that and take half of all products once more.
#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "fasa_chunk.cuh"
#include "fasa_tcgen05.cuh"

namespace fasa {
namespace {

constexpr int CB_NT = 384;           // 8 warps of rows, one of instructions, one of copies, two at rest
constexpr int CB_ROWS = 8;
constexpr uint32_t TM = 0;           // where tensor memory begins, which a block takes whole
constexpr int CB_K = CHUNK_TILE_BF16;
constexpr float CB_SLACK = 8.f;      // powers of two that a row's maximum may run ahead of m

template <int D>
struct CbPlan {
  static constexpr int HALVES = D / 64;                  // 64-column slabs of a row
  static constexpr int SLAB = 128 * 128;                 // bytes of one
  static constexpr int TILE = HALVES * SLAB;             // Q of 128 rows, K or V of 128 slots
  static constexpr int STAGES = D == 128 ? 4 : 8;        // K and V in turn
  static constexpr int OFF_RING = 2 * TILE;
  static constexpr int OFF_BAR = OFF_RING + STAGES * TILE;
  static constexpr int BARS = 2 * STAGES + 2 + 8 + 1;
  static constexpr int OFF_MISC = OFF_BAR + BARS * 8;    // tensor memory's address, dead
  static constexpr int OFF_SCAN = OFF_MISC + 16;          // (and whether a unit's V was not finite)
  static constexpr int OFF_TURN = (OFF_SCAN + CB_NT / 32 * 8 + 15) / 16 * 16;  // results on their way out, 2 KB a warp
  static constexpr int OFF_SEQ = OFF_TURN + CB_ROWS * 2048;
  static constexpr int bytes(int B) { return 1024 + OFF_SEQ + (B + 1) * 8; }
  static_assert(bytes(PAGED_MAX_BATCH) <= 232448, "the largest batch fits");
};

// The tiles of slots [f0, f1) of a unit that tile w of its rows reads: up to e.
__device__ __forceinline__ int row_tile_end(const ChunkParams& p, const ChunkUnit& u, int w, int f0, int f1) {
  const int TQ = 128 / p.G, j0 = (2 * u.i + w) * TQ;
  if (j0 >= u.q.n) return f0;
  const int see = u.q.len - u.q.n + min(j0 + TQ, u.q.n);
  return max(f0, min(f1, see > 0 ? (see + CB_K - 1) / CB_K : 0));
}

// Clears what a tile of V (128 rows at `tile`) brings to rows that do not see it: rows n .. 127,
// which hold anything (up to the pages' end; what lies behind that was not copied and is 0), and
// elements of rows r0 .. n - 1 that are not finite.  A warp; whether there were any.  A function
// of its own (eight prompts 314 us; inlined among the matrix instructions 326, without any of
// it 310); it has to do with the 56 registers of its warp.
template <int D>
__device__ __noinline__ bool clear_unseen(uint32_t tile, int r0, int n) {
  using P = CbPlan<D>;
  constexpr int CH = P::HALVES * 8, RS = 32 / CH;  // 16-byte chunks of a row, rows at a time
  const int lane = threadIdx.x & 31;
  const uint32_t place = tile + (lane % CH >> 3) * P::SLAB + lane / CH * 128 + ((lane & 7) << 4);
#pragma unroll 8
  for (int r = n; r < CB_K; r += RS)
    if (r + lane / CH < CB_K)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(place + r * 128), "r"(0) : "memory");
  bool found = false;
#pragma unroll 4
  for (int r = r0; r < n; r += RS) {
    uint32_t x[4] = {0u, 0u, 0u, 0u}, f[4];
    if (r + lane / CH < n)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                   : "r"(place + r * 128));
#pragma unroll
    for (int y = 0; y < 4; ++y) f[y] = ((x[y] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;  // (no carry)
    if (f[0] | f[1] | f[2] | f[3]) {
      found = true;
#pragma unroll
      for (int y = 0; y < 4; ++y) x[y] &= ~((f[y] >> 15) * 0xffffu);
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(place + r * 128), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                   "r"(x[3])
                   : "memory");
    }
  }
  fence_proxy_async();
  return __any_sync(0xffffffffu, found);
}

template <int D>
__global__ void __launch_bounds__(CB_NT, 1)
    chunk_bf16_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using P = CbPlan<D>;
  constexpr int S = P::STAGES;
  extern __shared__ __align__(16) char raw[];
  char* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t base = smem_u32(sm), ring = base + P::OFF_RING, bars = base + P::OFF_BAR;
  const uint32_t full = bars, empty = bars + 8 * S, q_full = bars + 16 * S, q_empty = q_full + 8;
  const uint32_t s_full = q_full + 16, o_full = q_full + 32;  // of either tile of rows
  const uint32_t p_full = q_full + 48, drain = q_full + 80;          // of either half of its P
  volatile int* misc = reinterpret_cast<volatile int*>(sm + P::OFF_MISC);
  const int TQ = 128 / p.G, TU = 2 * TQ;
  if (warp == 0) tm_alloc(base + P::OFF_MISC, 512);
  if (tid == 32) {
    misc[1] = 0;
    for (int i = 0; i < S; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(drain, 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(s_full + 8 * w, 1);
      mbar_init(p_full + 16 * w, 4);
      mbar_init(p_full + 16 * w + 8, 4);
      mbar_init(o_full + 8 * w, 2);
    }
    fence_mbar_init();
  }
  // rows of Q that no copy writes stay zeros
  for (int i = tid; i < 2 * P::TILE / 16; i += CB_NT) reinterpret_cast<uint4*>(sm)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async();
  tm_before_sync();
  paged_wait();
  paged_go();
  const ChunkLine line = chunk_line<CB_NT>(p, reinterpret_cast<long long*>(sm + P::OFF_SEQ),
                                           reinterpret_cast<long long*>(sm + P::OFF_SCAN), TU, CB_K, CHUNK_UNIT_BF16, blockIdx.x == 0);
  tm_after_sync();
  const int parts = line.parts(p.parts), c = blockIdx.x;
  const Patience patience{misc + 1, p.status, p.wait_ns};
  int copies = 0, q_copies = 0;  // that the copying warp has issued
  if (tid == 0) note_none(p, c);
  if (tid == 0 && c == 0) *p.queue = 0;
  if (c < parts) {
    const long long y0 = line.part_begin(parts, c), y1 = line.part_begin(parts, c + 1);
    // (384 threads of 168 registers: 256 of 224 and 128 of 56)
    if (warp < CB_ROWS) more_registers<224>();
    else fewer_registers<56>();
    if (warp < CB_ROWS) {
      // ------------------------------------------------ softmax: rows of tile w
      const int w = warp >> 2, row = tid & 127;
      const uint32_t here = TM + ((uint32_t)(warp & 3) << 21);  // lanes 32 (warp % 4) ..
      const uint32_t st = here + 128 * w, ot = here + 256 + 128 * w;
      const float scale = p.scale;
      uint32_t s_phase = 0, o_phase = 0;
      segments(line, y0, y1, [&](const ChunkUnit& u, int f0, int f1, bool whole) {
        const ChunkSeq& q = u.q;
        if (tid == 0 && !whole) note_record(p, c, u, TU, f0, f1);
        const int e = row_tile_end(p, u, w, f0, f1), j0 = (2 * u.i + w) * TQ;
        const int j = j0 + row / p.G;
        const bool live = row < TQ * p.G && j < q.n;
        const int see = live ? q.len - q.n + j + 1 : 0;
        // which groups of 16 slots lie in the pool, a tile ahead
        const int* table = p.page_table + (size_t)u.b * p.max_pages;
        auto look_up = [&](int t) {
          const int slot = t * CB_K + 16 * lane;
          return lane < 8 && slot < q.len ? table[slot >> p.log2_page] : 0;
        };
        int page = f0 < e ? look_up(f0) : 0;
        float* keep = live && chunk_light(p, u.b, q) ? chunk_logits(p, u.b, u.h, q) + (size_t)row * p.T_pad : nullptr;
        float m = -INFINITY;
        uint64_t l2 = 0;  // two sums
        for (int t = f0; t < e; ++t) {
          const unsigned held = __ballot_sync(0xffffffffu, page >= 0 && page < p.n_pages);
          if (t + 1 < e) page = look_up(t + 1);
          if (!patience.wait(s_full + 8 * w, s_phase)) return false;
          s_phase ^= 1;
          tm_after_sync();
          uint32_t s[128];
          tm_ld32(st, s);
          tm_ld32(st + 32, s + 32);
          tm_ld32(st + 64, s + 64);
          tm_ld32(st + 96, s + 96);
          tm_wait_ld();
          tm_settle(s);
          const int lim = see - t * CB_K;  // of the tile's slots
          if (__any_sync(0xffffffffu, lim < CB_K && live) || held != 0xffffffffu) {
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (i >= lim || !(held >> (i >> 4) & 1u)) s[i] = 0xff800000u;  // -inf
          }
          if (keep) {
            float4* to = reinterpret_cast<float4*>(keep + t * CB_K);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              to[i] = make_float4(__uint_as_float(s[4 * i]) * scale, __uint_as_float(s[4 * i + 1]) * scale,
                                  __uint_as_float(s[4 * i + 2]) * scale, __uint_as_float(s[4 * i + 3]) * scale);
          }
          float mx[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = __uint_as_float(s[i]);
#pragma unroll
          for (int i = 4; i < 128; i += 4)
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], __uint_as_float(s[i + k]));
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
          if (__any_sync(0xffffffffu, top > m + CB_SLACK)) {
            const float mn = top > m + CB_SLACK ? top : m;
            const float a = mn == -INFINITY ? 1.f : ex2(m - mn);
            m = mn;
            const uint64_t a2 = pair_of(a, a);
            l2 = mul2(l2, a2);
            if (t > f0) {  // (S of this tile was issued behind the last P V: O is at rest)
#pragma unroll
              for (int k = 0; k < D; k += 32) {
                uint32_t o[32];
                tm_ld32(ot + k, o);
                tm_wait_ld();
                tm_settle(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
                tm_st32(ot + k, o);
              }
            }
          }
          const float ms = m == -INFINITY ? 0.f : -m;
          const uint64_t scale2 = pair_of(scale, scale), ms2 = pair_of(ms, ms);
          // by halves: the tensor cores begin with the first
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t out[32];
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float x0, x1;
              unpair(fma2(pair_of(__uint_as_float(s[64 * h + 2 * i]), __uint_as_float(s[64 * h + 2 * i + 1])), scale2, ms2), x0, x1);
              x0 = ex2(x0);
              x1 = ex2(x1);
              sum[i & 1] = add2(sum[i & 1], pair_of(x0, x1));
              out[i] = pack_bf16(x0, x1);
            }
            l2 = add2(l2, add2(sum[0], sum[1]));
            tm_st32(st + 32 * h, out);
            tm_wait_st();
            tm_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + 16 * w + 8 * h);
          }
        }
        // ------------------------------------------------ the rows' results
        float la, lb;
        unpair(l2, la, lb);
        const float l = la + lb;
        if (f0 < e) {
          if (!patience.wait(o_full + 8 * w, o_phase)) return false;
          o_phase ^= 1;
          tm_after_sync();
        }
        const int r = w * TQ * p.G + row;  // of the unit
        const ChunkRow at(p, u, TU, r);
        float* rec = chunk_record(p, D, c, f0 > 0 ? 0 : 1);
        // Through shared memory, 64 bytes of a row at a time, so that four lanes write a row's
        // together: a store of 32 rows takes 32 turns, of eight rows eight.
        const unsigned alive = __ballot_sync(0xffffffffu, live);
        const long long mine = whole ? (long long)at.out(p, D) * 2 : (long long)r * D * 4;  // this row's place, bytes
        char* to[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          to[i] = (whole ? static_cast<char*>(p.out) : reinterpret_cast<char*>(rec)) +
                  __shfl_sync(0xffffffffu, mine, 8 * i + (lane >> 2)) + 16 * (lane & 3);
        const uint32_t turn = base + P::OFF_TURN + warp * 2048;
        auto send = [&](const uint32_t (&x)[16], int byte) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(turn + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)),
                         "r"(x[4 * i]), "r"(x[4 * i + 1]), "r"(x[4 * i + 2]), "r"(x[4 * i + 3])
                         : "memory");
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 8 * i + (lane >> 2);
            uint4 v;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(turn + row * 64 + (((lane & 3) ^ (row >> 1 & 3)) << 4))
                         : "memory");
            if (alive >> row & 1u) *reinterpret_cast<uint4*>(to[i] + byte) = v;
          }
          __syncwarp();
        };
        const float inv = l > 0.f ? 1.f / l : 0.f;
        uint32_t o[D];
        if (f0 < e) {
#pragma unroll
          for (int k = 0; k < D; k += 32) tm_ld32(ot + k, o + k);
          tm_wait_ld();
          tm_settle(o);
        } else {
#pragma unroll
          for (int i = 0; i < D; ++i) o[i] = 0u;
        }
#pragma unroll
        for (int k = 0; k < D; k += 32) {
          uint32_t x[16];
          if (whole) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              x[i] = pack_bf16(__uint_as_float(o[k + 2 * i]) * inv, __uint_as_float(o[k + 2 * i + 1]) * inv);
            send(x, 2 * k);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = o[k + i];
            send(x, 4 * k);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = o[k + 16 + i];
            send(x, 4 * k + 64);
          }
        }
        tm_before_sync();  // (the next unit's first P is behind this)
        if (live && whole && p.weight) p.lse[at.lse(p)] = chunk_lse(m, l);
        if (live && !whole) {
          rec[(size_t)p.rows * D + r] = m;
          rec[(size_t)p.rows * (D + 1) + r] = l;
        }
        if (f0 < e && misc[2 + w]) {  // (the results are stored by other lanes of the warp)
          __syncwarp();
          const int s0 = max(partly_seen(u, TU).x, f0 * CB_K), s1 = min(see, f1 * CB_K);
          if (live && whole)
            add_not_finite<__nv_bfloat16>(p, u.b, u.h, s0, s1, 0, D, D, static_cast<__nv_bfloat16*>(p.out) + at.out(p, D));
          else if (live)
            add_not_finite<__nv_bfloat16>(p, u.b, u.h, s0, s1, 0, D, D, rec + (size_t)r * D);
        }
        return true;
      });
    } else if (warp == CB_ROWS) {
      // ------------------------------------------------ matrix instructions
      constexpr uint32_t kind_s = mma_bf16_kind(CB_K, false), kind_o = mma_bf16_kind(D, true);
      uint32_t q_phase = 0, p_phase[2] = {0, 0};
      int k = 0;  // tiles of the ring so far
      auto at = [&](int i) { return ring + (i % S) * P::TILE; };
      auto landed = [&](int i) { return patience.wait(full + 8 * (i % S), (i / S) & 1); };
      // (descriptors count 16 bytes)
      const uint64_t q_tile = mma_operand(base, 0), k_tile = mma_operand(ring, 0), v_tile = mma_operand(ring, P::SLAB);
      auto scores = [&](int w, int i) {  // S of row tile w with the K of ring tile i
        const uint64_t a = q_tile + (w * P::TILE >> 4), b = k_tile + ((uint32_t)(i % S) * P::TILE >> 4);
        if (elected()) {
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            const uint32_t off = ((x >> 2) * P::SLAB + (x & 3) * 32) >> 4;
            mma_ss(TM + 128 * w, a + off, b + off, kind_s, x > 0);
          }
          mma_commit(s_full + 8 * w);
        }
      };
      auto free_tile = [&](uint32_t bar) {
        if (elected()) mma_commit(bar);
      };
      segments(line, y0, y1, [&](const ChunkUnit& u, int f0, int f1, bool) {
        const ChunkSeq& q = u.q;
        const int e0 = row_tile_end(p, u, 0, f0, f1), e1 = row_tile_end(p, u, 1, f0, f1);
        const int e[2] = {e0, e1}, end = max(e0, e1);
        if (f0 == end) return true;
        const int2 partly = partly_seen(u, TU);
        bool odd = false;
        if (!patience.wait(q_full, q_phase)) return false;
        q_phase ^= 1;
        if (!landed(k)) return false;
#pragma unroll
        for (int w = 0; w < 2; ++w)
          if (f0 < e[w]) scores(w, k);
        free_tile(empty + 8 * (k % S));
        if (f0 + 1 == end) free_tile(q_empty);
        for (int t = f0; t < end; ++t, k += 2) {
          if (!landed(k + 1)) return false;
          if ((t + 1) * CB_K > partly.x) {
            odd = clear_unseen<D>(at(k + 1), max(0, partly.x - t * CB_K), min(CB_K, partly.y - t * CB_K)) || odd;
            __syncwarp();
          }
          const bool more = t + 1 < end;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (t < e[w]) {
              const uint64_t b = v_tile + ((uint32_t)((k + 1) % S) * P::TILE >> 4);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (!patience.wait(p_full + 16 * w + 8 * h, p_phase[w])) return false;
                tm_after_sync();
                if (elected()) {
#pragma unroll
                  for (int x = 4 * h; x < 4 * h + 4; ++x)
                    mma_ts(TM + 256 + 128 * w, TM + 128 * w + 8 * x, b + (2048 * x >> 4), kind_o, t > f0 || x > 0);
                  if (h == 1 && t + 1 == e[w]) {
                    misc[2 + w] = odd;  // (the rows' last P came: they have read the last unit's)
                    mbar_arrive(o_full + 8 * w);
                    mma_commit(o_full + 8 * w);
                  }
                }
              }
              p_phase[w] ^= 1;
            }
            if (w == 1) free_tile(empty + 8 * ((k + 1) % S));
            if (more && w == 0 && !landed(k + 2)) return false;
            if (t + 1 < e[w]) scores(w, k + 2);
          }
          if (more) free_tile(empty + 8 * ((k + 2) % S));
          if (t + 2 == end) free_tile(q_empty);
        }
        return true;
      });
    } else if (warp == CB_ROWS + 1) {
      // ------------------------------------------------ copies
      const int box = min(1 << p.log2_page, 128), per = 128 / box;  // rows of a copy, copies of a slab
      const int none = (int)((long long)p.n_pages * p.Hkv << p.log2_page);  // a row behind the pool: zeros
      const int mine = lane / P::HALVES, half = lane % P::HALVES;
      uint32_t q_phase = 1;
      int& k = copies;
      int n_tile = 0;
      fence_proxy_async_global();  // (a kernel before this one may have stored what is copied)
      segments(line, y0, y1, [&](const ChunkUnit& u, int f0, int f1, bool) {
        const ChunkSeq& q = u.q;
        const int end = max(row_tile_end(p, u, 0, f0, f1), row_tile_end(p, u, 1, f0, f1));
        if (f0 == end) return true;
        const int first = q.first + u.i * TU;
        if (!patience.wait(q_empty, q_phase)) return false;
        q_phase ^= 1;
        ++q_copies;
        if (lane == 0) mbar_arrive_expect_tx(q_full, 2 * P::HALVES * TQ * p.G * 128);
        __syncwarp();
        if (lane < 2 * P::HALVES) {
          const int w = lane / P::HALVES;
          tma_3d(base + w * P::TILE + half * P::SLAB, &qmap, 64 * half, u.h * p.G, first + w * TQ, q_full);
        }
        __syncwarp();
        if (u.begin + u.cost < y1) {  // the next unit's Q into L2: it is waited for between the units
          ChunkUnit v = u;
          v.next(line);
          const int token = v.q.first + v.i * TU + lane / P::HALVES * TQ;
          if (lane < 2 * P::HALVES && token < p.n_tokens) tma_prefetch_3d(&qmap, 64 * half, v.h * p.G, token);
        }
        const int* table = p.page_table + (size_t)u.b * p.max_pages;
        auto look_up = [&](int t) {
          const int slot = t * CB_K + mine * box;
          return mine < per && slot < q.len ? table[slot >> p.log2_page] : -1;
        };
        int page = look_up(f0);
        for (int t = f0; t < end; ++t) {
          const int slot = t * CB_K + mine * box;
          long long row = paged_row(page, p.n_pages, p.Hkv, u.h, p.log2_page, slot);
          if (row < 0 && mine < per && slot < q.len) atomicOr(p.status, 1);
          if (row < 0) row = none;
          if (t + 1 < end) page = look_up(t + 1);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++k) {
            const int st = k % S;
            if (!patience.wait(empty + 8 * st, (k / S & 1) ^ 1)) return false;
            if (lane == 0) mbar_arrive_expect_tx(full + 8 * st, P::TILE);
            __syncwarp();
            if (mine < per && n_tile != p.drop_tile)  // (test hook: copies that never come)
              tma_2d(ring + st * P::TILE + half * P::SLAB + mine * box * 128, kv ? &vmap : &kmap, 64 * half, (int)row,
                     full + 8 * st);
            __syncwarp();
          }
          ++n_tile;
        }
        return true;
      });
    }
  }
  // After a wait that ran out, no copy may land in memory of a block that is gone, nor may
  // matrix instructions be under way when tensor memory goes back.
  __syncthreads();
  if (misc[1] && warp == CB_ROWS) {
    if (elected()) mma_commit(drain);
    if (!mbar_wait_bounded(drain, 0, 8 * p.wait_ns) && lane == 0) atomicOr(p.status, 4);
  } else if (misc[1] && warp == CB_ROWS + 1) {
    bool all = q_copies == 0 || mbar_wait_bounded(q_full, (q_copies - 1) & 1, 8 * p.wait_ns);
    for (int i = max(0, copies - S); i < copies; ++i)
      all = mbar_wait_bounded(full + 8 * (i % S), (i / S) & 1, 8 * p.wait_ns) && all;
    if (!all && lane == 0) atomicOr(p.status, 4);
  }
  __syncthreads();
  if (warp == 0) tm_free(TM, 512);
}

// ------------------------------------------------------------------ weights
// weight_t += sum over the rows that see slot t of 2^(scale S - log-sum of the row).  A
// unit is 256 slots of a (sequence, KV head): two tiles of K as rows of S^T = K Q^T, the
// rows of Q 128 at a time as its columns (K in tensor memory, Q in shared memory), so that a
// thread adds what one slot gets, in the rows' order.
constexpr int CW_NT = 640;           // 16 warps of slots, one of instructions, one of copies, two at rest
constexpr int CW_ROWS = 16;
constexpr int CW_S = 3;              // tiles of S in tensor memory, of 128 columns, behind the two tiles of K

// Two warps with the two halves of the same rows' columns.
struct Pair {
  int id, half;
  float* at;  // shared memory, 32 floats
  // Whether either says so.  Also a barrier.
  __device__ bool either(bool x) const { return named_bar_or(id, 64, x); }
  // op(x, the other's x), the same in both: in a fixed order.
  template <class F>
  __device__ float join(float x, F&& op) const {
    float* mine = at + (threadIdx.x & 31);
    if (half) *mine = x;
    named_bar_sync(id, 64);
    if (!half) *mine = x = op(x, *mine);
    named_bar_sync(id, 64);
    return half ? *mine : x;
  }
};

constexpr int CW_LSE = 4;             // tiles of Q whose rows' log-sums are there

template <int D>
struct CwPlan {
  using A = CbPlan<D>;
  static constexpr int STAGES = 6 * A::STAGES / 4;  // of the ring: a unit's two tiles of K, then its tiles of Q
  static constexpr int TILE = A::TILE;
  static constexpr int OFF_LSE = STAGES * TILE;
  static constexpr int OFF_BAR = OFF_LSE + CW_LSE * 128 * 4;
  static constexpr int BARS = 2 * STAGES + 2 * CW_LSE + 2 + 8 + CW_S + 1 + 4;
  static constexpr int OFF_MISC = OFF_BAR + BARS * 8;
  static constexpr int OFF_PAIR = (OFF_MISC + 16 + 15) / 16 * 16;
  static constexpr int OFF_LINE = OFF_PAIR + CW_ROWS / 2 * 128;
  static constexpr int bytes(int B) { return 1024 + OFF_LINE + (3 * B + 3) * 4; }
  static_assert(bytes(PAGED_MAX_BATCH) <= 232448, "the largest batch fits");
};

// A place of the ring.
template <int S>
struct RingAt {
  int st = 0;
  uint32_t phase = 0;
  __device__ void next() {
    if (++st == S) {
      st = 0;
      phase ^= 1;
    }
  }
};

// What a slot gets of 64 columns of S at `at`, which are then free (`done`): those that `there` says
// are rows, and of them those that `sees` says see the slot.  l: the rows' negative log-sums, maybe
// NaN, so that a row that does not see the slot is masked behind the sum with it.
template <class There, class Sees>
__device__ __forceinline__ float columns_sum(uint32_t at, uint32_t done, const float* l, float scale, There&& there, Sees&& sees) {
  uint32_t s[64];
  tm_ld32(at, s);
  tm_ld32(at + 32, s + 32);
  tm_wait_ld();
  tm_settle(s);
  tm_before_sync();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(done);
#pragma unroll
  for (int x = 0; x < 64; ++x)
    if (!there(x)) s[x] = 0xff800000u;  // -inf
  const uint64_t scale2 = pair_of(scale, scale);
  uint64_t sum[2] = {0, 0};
#pragma unroll
  for (int x = 0; x < 16; ++x) {
    const float4 y = reinterpret_cast<const float4*>(l)[x];
    float a[4];
    unpair(fma2(pair_of(__uint_as_float(s[4 * x]), __uint_as_float(s[4 * x + 1])), scale2, pair_of(y.x, y.y)), a[0], a[1]);
    unpair(fma2(pair_of(__uint_as_float(s[4 * x + 2]), __uint_as_float(s[4 * x + 3])), scale2, pair_of(y.z, y.w)), a[2], a[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (!sees(4 * x + e)) a[e] = -INFINITY;
    sum[0] = add2(sum[0], pair_of(ex2(a[0]), ex2(a[1])));
    sum[1] = add2(sum[1], pair_of(ex2(a[2]), ex2(a[3])));
  }
  float a, b;
  unpair(add2(sum[0], sum[1]), a, b);
  return a + b;
}
// A tile whose rows end, or of which some do not see all of the warp's slots: few.  A function of
// its own: a prompt of 16K tokens with weights 2022 us, 2060 with both kinds of sums in line (2014
// with the mask ahead of the log-sum, where NaN reaches slots that its row does not see).
__device__ __noinline__ static float edge_sum(uint32_t at, uint32_t done, const float* l, float scale, int lo, int rows) {
  return columns_sum(at, done, l, scale, [](int) { return true; }, [&](int x) { return x >= lo && x < rows; });
}

template <int D>
__global__ void __launch_bounds__(CW_NT, 1)
    chunk_weight_bf16_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap qmap,
                             const __grid_constant__ CUtensorMap kmap) {
  using P = CwPlan<D>;
  using A = CbPlan<D>;
  constexpr int S = P::STAGES;
  extern __shared__ __align__(16) char raw[];
  char* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t ring = smem_u32(sm), full = ring + P::OFF_BAR, empty = full + 8 * S;
  const uint32_t lse_full = empty + 8 * S, lse_empty = lse_full + 8 * CW_LSE, k_go = lse_empty + 8 * CW_LSE;
  const uint32_t k_here = k_go + 8, t_full = k_go + 16, t_empty = t_full + 64, drain = t_empty + 8 * CW_S;
  const uint32_t u_full = drain + 8, u_empty = drain + 24;
  volatile int* misc = reinterpret_cast<volatile int*>(sm + P::OFF_MISC);
  float* lse = reinterpret_cast<float*>(sm + P::OFF_LSE);
  int* before = reinterpret_cast<int*>(sm + P::OFF_LINE);
  const int TQ = 128 / p.G;
  if (warp == 0) tm_alloc(ring + P::OFF_MISC, 512);
  if (tid == 32) {
    misc[1] = 0;
    for (int i = 0; i < S; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < CW_LSE; ++i) {
      mbar_init(lse_full + 8 * i, 1);
      mbar_init(lse_empty + 8 * i, CW_ROWS);
    }
    mbar_init(k_go, 1);
    mbar_init(k_here, CW_ROWS);
    // (a barrier that its waiters may find two phases on tells them nothing: those of full
    // tiles of S are each row tile's own, and more than there are tiles)
    for (int i = 0; i < 8; ++i) mbar_init(t_full + 8 * i, 1);
    for (int i = 0; i < CW_S; ++i) mbar_init(t_empty + 8 * i, 8);
    mbar_init(drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(u_full + 8 * i, 1);
      mbar_init(u_empty + 8 * i, CW_ROWS + 1);
    }
    fence_mbar_init();
  }
  tm_before_sync();
  paged_go();
  paged_wait();
  weight_line<CW_NT, 256>(p, before, reinterpret_cast<int3*>(sm + P::OFF_PAIR), TQ);
  tm_after_sync();
  if (p.logits) weight_light<CW_NT>(p, before + 2 * (p.B + 1));
  const Patience patience{misc + 1, p.status, p.wait_ns};
  int issued = 0;  // copies
  // f(unit) for each unit of this block, in order, as the copying warp takes them.  came(x):
  // whether the unit came for all warps that f has wait for each other: one that gives up
  // alone would leave the others at a barrier without a limit.
  auto units = [&](auto&& came, auto&& f) {
    for (int i = 0;; ++i) {
      if (!came(patience.wait(u_full + 8 * (i & 1), i >> 1 & 1))) return;
      const int x = misc[2 + (i & 1)];
      __syncwarp();
      if (lane == 0) mbar_arrive(u_empty + 8 * (i & 1));
      WeightUnit u;
      if (!weight_unit<256>(p, before, x, u) || !f(u)) return;
    }
  };
  // (640 threads of 96 registers: 512 of 104 and 128 of 64)
  if (warp < CW_ROWS) more_registers<104>();
  else fewer_registers<64>();
  if (warp < CW_ROWS) {
    // -------------------------------------------------- a slot to a thread, half of Q's rows
    const int w = warp >> 3, half = (warp >> 2) & 1, row = tid & 127;
    const Pair pair{1 + (warp >> 3) * 4 + (warp & 3), half,
                    reinterpret_cast<float*>(sm + P::OFF_PAIR) + 32 * ((warp >> 3) * 4 + (warp & 3))};
    const uint32_t here = TM + ((uint32_t)(warp & 3) << 21);
    const float scale = p.scale;
    int at_k = 0;  // place of the next unit's K in the ring
    uint32_t k_phase = 0;
    int k = 0, n_s = 0, own = 0;  // Q tiles, S tiles, and those of these rows, so far
    units([&](bool x) { return !pair.either(!x); }, [&](const WeightUnit& u) {
      const int slot = u.t0 + 128 * w + row, from = u.from(0, TQ), mine = u.from(128 * w, TQ), tiles = u.tiles(TQ);
      if (from >= tiles) return true;
      int page = -1;
      if (slot < u.q.len) page = p.page_table[(size_t)u.b * p.max_pages + (slot >> p.log2_page)];
      float* weight = p.weight + ((size_t)u.b * p.Hkv + u.h) * p.T_cap + slot;
      const bool live = page >= 0 && page < p.n_pages;
      const float old = live && !half ? *weight : 0.f;
      float total = 0.f;
      // K from shared to tensor memory, a row to a thread: the matrix instructions then read
      // Q alone from shared memory, whose bandwidth would bound them
      bool ok = patience.wait(k_go, k_phase);
      k_phase ^= 1;
      {
        const uint32_t tile = ring + (uint32_t)((at_k + w) % S) * P::TILE;
        at_k = (at_k + 2 + tiles - from) % S;  // (behind the tiles of Q)
        constexpr int CH = D / 16;  // 16-byte chunks of half a row
        uint32_t x[4 * CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int ch = CH * half + i;
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[4 * i]), "=r"(x[4 * i + 1]), "=r"(x[4 * i + 2]), "=r"(x[4 * i + 3])
                       : "r"(tile + (ch >> 3) * A::SLAB + row * 128 + (((ch & 7) ^ (row & 7)) << 4))
                       : "memory");
        }
        if constexpr (D == 128) tm_st32(here + 64 * w + 32 * half, x);
        else tm_st16(here + 32 * w + 16 * half, x);
        tm_wait_st();
        tm_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_here);
      }
      const int second = u.from(128, TQ);
      for (int i = from; ok && i < tiles; ++i, ++k) {
        const int st = k % CW_LSE;
        ok = patience.wait(lse_full + 8 * st, (k / CW_LSE) & 1);
        if (!ok) break;
        const int buf = (n_s + w) % CW_S;
        n_s += i >= second ? 2 : 1;
        if (i >= mine) {
          // the rows of this tile that there are, and of them the first that sees the slot
          const int rows = min(TQ, u.q.n - i * TQ) * p.G - 64 * half, lo = (slot - (u.q.len - u.q.n) - i * TQ) * p.G - 64 * half;
          const bool edge = rows < TQ * p.G - 64 * half || __any_sync(0xffffffffu, lo > 0);
          ok = patience.wait(t_full + 32 * w + 8 * (own & 3), own >> 2 & 1);
          if (!ok) break;
          ++own;
          tm_after_sync();
          const uint32_t at = here + 128 * (1 + buf) + 64 * half, done = t_empty + 8 * buf;
          const float* l = lse + 128 * st + 64 * half;  // (negative log-sums)
          if (edge) {
            total += edge_sum(at, done, l, scale, lo, rows);
          } else {
            // (columns behind a tile's rows hold anything; a tile has 125 rows or more)
            total += columns_sum(at, done, l, scale, [&](int x) { return x < 61 || x < rows; }, [](int) { return true; });
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(lse_empty + 8 * st);
      }
      if (pair.either(!ok)) return false;
      total = pair.join(total, [](float a, float b) { return a + b; });
      if (live && !half && total != 0.f) *weight = old + total;
      return true;
    });
  } else if (warp == CW_ROWS) {
    // -------------------------------------------------- matrix instructions
    constexpr uint32_t kind = mma_bf16_kind(128, false);
    const uint64_t q_tile = mma_operand(ring, 0);  // (descriptors count 16 bytes)
    RingAt<S> at;
    uint32_t k_phase = 0;
    int n_s = 0, own[2] = {0, 0};
    units([](bool x) { return x; }, [&](const WeightUnit& u) {
      const int from[2] = {u.from(0, TQ), u.from(128, TQ)}, tiles = u.tiles(TQ);
      if (from[0] >= tiles) return true;
      int k_at[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        k_at[w] = at.st;
        if (!patience.wait(full + 8 * at.st, at.phase)) return false;
        at.next();
      }
      if (lane == 0) mbar_arrive(k_go);
      __syncwarp();
      if (!patience.wait(k_here, k_phase)) return false;
      k_phase ^= 1;
      if (lane < 2) mbar_arrive(empty + 8 * (lane ? k_at[1] : k_at[0]));
      __syncwarp();
      tm_after_sync();
      for (int i = from[0]; i < tiles; ++i, at.next()) {
        const int st = at.st;
        if (!patience.wait(full + 8 * st, at.phase)) return false;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (i < from[w]) continue;
          const int b = n_s % CW_S;
          if (!patience.wait(t_empty + 8 * b, (n_s / CW_S & 1) ^ 1)) return false;
          ++n_s;
          tm_after_sync();
          const uint64_t columns = q_tile + ((uint32_t)st * P::TILE >> 4);
          if (elected()) {
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
              const uint32_t off = ((x >> 2) * A::SLAB + (x & 3) * 32) >> 4;
              mma_ts(TM + 128 * (1 + b), TM + D / 2 * w + 8 * x, columns + off, kind, x > 0);
            }
            mma_commit(t_full + 32 * w + 8 * (own[w] & 3));
          }
          ++own[w];
        }
        if (elected()) mma_commit(empty + 8 * st);
      }
      return true;
    });
  } else if (warp == CW_ROWS + 1) {
    // -------------------------------------------------- copies
    const int box = min(1 << p.log2_page, 128), per = 128 / box;
    const int none = (int)((long long)p.n_pages * p.Hkv << p.log2_page);
    const int half = lane % A::HALVES, mine = lane / A::HALVES;
    RingAt<S> at;
    int k = 0;
    fence_proxy_async_global();
    auto copy = [&](const WeightUnit& u) {
      const int from = u.from(0, TQ), tiles = u.tiles(TQ);
      if (from >= tiles) return true;
      int row[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int slot = u.t0 + 128 * w + mine * box;
        long long x = -1;
        if (mine < per && slot < u.q.len)
          x = paged_row(p.page_table[(size_t)u.b * p.max_pages + (slot >> p.log2_page)], p.n_pages, p.Hkv, u.h,
                        p.log2_page, slot);
        row[w] = x < 0 ? none : (int)x;
      }
#pragma unroll
      for (int w = 0; w < 2; ++w, at.next()) {
        if (!patience.wait(empty + 8 * at.st, at.phase ^ 1)) return false;
        if (lane == 0) mbar_arrive_expect_tx(full + 8 * at.st, P::TILE);
        __syncwarp();
        if (mine < per)
          tma_2d(ring + at.st * P::TILE + half * A::SLAB + mine * box * 128, &kmap, 64 * half, row[w], full + 8 * at.st);
        __syncwarp();
        ++issued;
      }
      for (int i = from; i < tiles; ++i, ++k, at.next()) {
        const int rows = min(TQ, u.q.n - i * TQ) * p.G, sl = k % CW_LSE;
        const float* from_lse = p.lse + ((size_t)u.h * p.n_tokens + u.q.first + i * TQ) * p.G;
        float l[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) l[x] = lane + 32 * x < rows ? -ld_cg(from_lse + lane + 32 * x) : -INFINITY;
        if (!patience.wait(lse_empty + 8 * sl, (k / CW_LSE & 1) ^ 1)) return false;
#pragma unroll
        for (int x = 0; x < 4; ++x) lse[128 * sl + lane + 32 * x] = l[x];
        __syncwarp();
        if (lane == 0) mbar_arrive(lse_full + 8 * sl);
        if (!patience.wait(empty + 8 * at.st, at.phase ^ 1)) return false;
        if (lane == 0) mbar_arrive_expect_tx(full + 8 * at.st, A::HALVES * TQ * p.G * 128);
        __syncwarp();
        if (lane < A::HALVES)
          tma_3d(ring + at.st * P::TILE + lane * A::SLAB, &qmap, 64 * lane, u.h * p.G, u.q.first + i * TQ, full + 8 * at.st);
        __syncwarp();
        ++issued;
      }
      return true;
    };
    int x = blockIdx.x;  // (the first unit is the block's own; the queue counts those behind)
    for (int i = 0;; ++i) {
      if (!patience.wait(u_empty + 8 * (i & 1), (i >> 1 & 1) ^ 1)) break;
      if (lane == 0) {
        misc[2 + (i & 1)] = x;
        mbar_arrive(u_full + 8 * (i & 1));
      }
      __syncwarp();
      WeightUnit u;
      if (!weight_unit<256>(p, before, x, u)) break;
      int next = 0;  // (on its way while this one is copied)
      if (lane == 0) next = gridDim.x + atomicAdd(p.queue, 1);
      if (!copy(u)) break;
      x = __shfl_sync(0xffffffffu, next, 0);
    }
  }
  __syncthreads();  // (and then as above)
  if (misc[1] && warp == CW_ROWS) {
    if (elected()) mma_commit(drain);
    if (!mbar_wait_bounded(drain, 0, 8 * p.wait_ns) && lane == 0) atomicOr(p.status, 4);
  } else if (misc[1] && warp == CW_ROWS + 1) {
    bool all = true;
    for (int i = max(0, issued - S); i < issued; ++i)
      all = mbar_wait_bounded(full + 8 * (i % S), (i / S) & 1, 8 * p.wait_ns) && all;
    if (!all && lane == 0) atomicOr(p.status, 4);
  }
  __syncthreads();
  if (warp == 0) tm_free(TM, 512);
}

template <int D>
cudaError_t launch(const ChunkParams& p, cudaStream_t s) {
  using P = CbPlan<D>;
  static std::atomic<unsigned long long> allowed{0};  // devices that were told of the shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (!(allowed.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(chunk_bf16_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::bytes(PAGED_MAX_BATCH));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(chunk_weight_bf16_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               CwPlan<D>::bytes(PAGED_MAX_BATCH));
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_release);
  }
  const int TQ = 128 / p.G;
  CUtensorMap qm, km, vm;
  const cuuint64_t qd[3] = {D, (cuuint64_t)p.Hq, (cuuint64_t)p.n_tokens}, qs[2] = {D * 2, (cuuint64_t)p.Hq * D * 2};
  const cuuint32_t qb[3] = {64, (cuuint32_t)p.G, (cuuint32_t)TQ};
  e = tensor_map(&qm, p.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, qd, qs, qb);
  const cuuint64_t kd[2] = {D, ((cuuint64_t)p.n_pages * p.Hkv) << p.log2_page}, ks[1] = {D * 2};
  const cuuint32_t kb[2] = {64, (cuuint32_t)std::min(1 << p.log2_page, 128)};
  if (e == cudaSuccess) e = tensor_map(&km, p.k_pages, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, kd, ks, kb);
  if (e == cudaSuccess) e = tensor_map(&vm, p.v_pages, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, kd, ks, kb);
  if (e == cudaSuccess) e = paged_behind(chunk_bf16_kernel<D>, p.parts, CB_NT, P::bytes(p.B), 0, s, p, qm, km, vm);
  if (e == cudaSuccess) e = launch_chunk_join<__nv_bfloat16, D>(p, s);
  if (e == cudaSuccess && p.weight)
    e = paged_behind(chunk_weight_bf16_kernel<D>, p.sms, CW_NT, CwPlan<D>::bytes(p.B), 0, s, p, qm, km);
  return e;
}

}  // namespace

cudaError_t launch_chunk_bf16(const ChunkParams& p, int head_dim, cudaStream_t s) {
  return head_dim == 128 ? launch<128>(p, s) : launch<64>(p, s);
}

}  // namespace fasa
