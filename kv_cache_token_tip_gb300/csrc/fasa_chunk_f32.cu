// Attention of chunks in fp32 on CUDA cores.  A block takes a part of the line of units
// (fasa_chunk_index.h): up to 128 rows (new tokens times the heads of their group), the
// slots 64 at a time.
//
// A thread has 8 rows and 4 slots of Z = Q K^T and 8 rows and D / 16 dims of O, its products
// two at a time (fma.f32x2: the instruction alone would fill the issue slots that the
// operands' loads need too).  A warp of its own copies (TMA boxes of a page's rows); no warp
// waits for another's rows, so that one's softmax is hidden by the others' products.  K of
// the next tile is on its way while P V is worked out, V while Q K^T is.  Bound by the
// products: two prompts of 1000 and 1500 tokens, 8 heads of 128 dims, 232 us, 36.6 TFLOP/s of
// visible pairs, half of the FMA rate.  O is summed a tile at a time and then over tiles: one
// after another, 217 us, but 16384 slots are off by 2.0e-6 of the result instead of 6e-7.
// (With such sums all warps in step and copying took 253 us, copies row by row, whose issue
// takes 3.5 us a tile, 227.)
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "fasa_cluster.cuh"
#include "fasa_chunk.cuh"
#include "fasa_tcgen05.cuh"

namespace fasa {
namespace {

constexpr int CF_NT = 256, CF_M = 128, CF_K = CHUNK_TILE_F32;

template <int D>
struct CfPlan {
  // Q, K, V as slabs of 32 dims, 128 bytes of a row each, in the 128-byte swizzle; P's rows
  // apart by four banks
  static constexpr int SLABS = D / 32, LP = CF_K + 4;
  static constexpr int Q_BYTES = CF_M * D * 4, K_BYTES = CF_K * D * 4;
  // attention: Q, K, V, P, which slots count (two tiles), barriers, the line
  static constexpr int OFF_K = Q_BYTES, OFF_V = OFF_K + K_BYTES, OFF_P = OFF_V + K_BYTES;
  static constexpr int OFF_HELD = OFF_P + CF_M * LP * 4;
  static constexpr int OFF_BAR = OFF_HELD + 24;
  static constexpr int OFF_SCAN = OFF_BAR + 7 * 8;
  static constexpr int OFF_LINE = OFF_SCAN + 12 * 8;
  static constexpr int bytes(int B) { return 1024 + OFF_LINE + (B + 1) * 8; }
  // weights: K, Q and its rows' log-sums twice, sums
  static constexpr int W_Q = K_BYTES, W_LSE = W_Q + 2 * Q_BYTES, W_SUM = W_LSE + 2 * CF_M * 4;
  static constexpr int W_ROWS = W_SUM + 16 * LP * 4, W_SCAN = W_ROWS + CF_K * 4, W_LINE = W_SCAN + CF_NT / 32 * 12;
  static constexpr int weight_bytes(int B) { return W_LINE + (3 * B + 3) * 4; }
  static_assert(bytes(PAGED_MAX_BATCH) <= 232448 && weight_bytes(PAGED_MAX_BATCH) <= 232448, "the largest batch fits");
};

// Pool rows of the slots t0 .. t0 + 63 of (b, h), -1 for those that do not count: a slot to a
// thread of the first 64.
__device__ __forceinline__ int slot_row(const ChunkParams& p, int b, int h, int t, int len, bool report) {
  if (t >= len) return -1;
  const int row = (int)paged_row(p.page_table[(size_t)b * p.max_pages + (t >> p.log2_page)], p.n_pages, p.Hkv, h, p.log2_page, t);
  if (row < 0 && report) atomicOr(p.status, 1);
  return row;
}

// Where 16-byte chunk c of row r lies in slabs of `rows` rows.
__device__ __forceinline__ int swizzled(int rows, int r, int c) { return (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4); }

// 64 rows of K, zeros for those that do not count.
template <int D>
__device__ __forceinline__ void fetch_slots(const void* pages, const int* rows, char* to) {
  constexpr int CH = D / 4;
#pragma unroll
  for (int i = threadIdx.x; i < CF_K * CH; i += CF_NT) {
    const int r = i / CH, c = i % CH, row = rows[r];
    cp_async16_zfill(smem_u32(to + swizzled(CF_K, r, c)), static_cast<const float*>(pages) + (size_t)max(row, 0) * D + 4 * c,
                     row >= 0 ? 16u : 0u);
  }
  cp_async_commit();
}

// Rows of a unit's queries: `count` of them from token `token` on, head group h; behind them the
// last one again: zeros times an infinite key would be NaN, and add that to a slot, where a row's
// copy, of weight 0, adds nothing unless the row itself makes the slot NaN.
template <int D>
__device__ __forceinline__ void fetch_queries(const ChunkParams& p, int token, int h, int count, char* to) {
  constexpr int CH = D / 4;
  const int all = (count + 15) / 16 * 16 * CH;  // (warps without rows read nothing)
#pragma unroll 4
  for (int i = threadIdx.x; i < all; i += CF_NT) {
    const int r = i / CH, c = i % CH, x = min(r, count - 1), j = x / p.G;
    const size_t from = ((size_t)(token + j) * p.Hq + h * p.G + x - j * p.G) * D + 4 * c;
    cp_async16(smem_u32(to + swizzled(CF_M, r, c)), static_cast<const float*>(p.q) + from);
  }
  cp_async_commit();
}

// z[i][j]: row 8 ty + i, slot tx + 16 j.  The even and the odd dims add up apart.
template <int D>
__device__ __forceinline__ void products(const char* q, const char* k, float (&z)[8][4]) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  uint64_t acc[8][4];
#pragma unroll
  for (int i = 0; i < 32; ++i) acc[i >> 2][i & 3] = 0;
  q += 8 * ty * 128;
  k += tx * 128;
#pragma unroll 1
  for (int slab = 0; slab < D / 32; ++slab, q += CF_M * 128, k += CF_K * 128) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      ulonglong2 b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const ulonglong2*>(k + 16 * 128 * j + ((c ^ (tx & 7)) << 4));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(q + i * 128 + ((c ^ i) << 4));
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fma2(a.y, b[j].y, fma2(a.x, b[j].x, acc[i][j]));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    float x, y;
    unpair(acc[i >> 2][i & 3], x, y);
    z[i >> 2][i & 3] = x + y;
  }
}

constexpr int CA_NT = 384;  // 8 warps of rows, one of copies, three at rest

template <int D>
__global__ void __launch_bounds__(CA_NT, 1)
    chunk_f32_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using P = CfPlan<D>;
  constexpr int E = D / 64;  // groups of 4 dims of a thread: 4 tx + 64 e ..
  extern __shared__ __align__(16) char raw[];
  char* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  char *qs = sm, *ks = sm + P::OFF_K, *vs = sm + P::OFF_V;
  float* ps = reinterpret_cast<float*>(sm + P::OFF_P);
  volatile unsigned* held = reinterpret_cast<unsigned*>(sm + P::OFF_HELD);  // two tiles' masks of slots that count
  volatile int* dead = reinterpret_cast<int*>(sm + P::OFF_HELD) + 4;
  volatile int* not_all_finite = dead + 1;  // V of the tile, where not all rows see it
  const uint32_t bars = smem_u32(sm + P::OFF_BAR);
  const uint32_t q_full = bars, q_empty = bars + 8, k_full = bars + 16, k_empty = bars + 24, v_full = bars + 32,
                 v_empty = bars + 40, v_raw = bars + 48;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), TU = CF_M / p.G;
  if (tid == 0) {
    *dead = 0;
    for (int i = 0; i < 7; ++i) mbar_init(bars + 8 * i, i & 1 ? CF_NT / 32 : 1);
    fence_mbar_init();
  }
  paged_wait();
  paged_go();
  const ChunkLine line = chunk_line<CA_NT>(p, reinterpret_cast<long long*>(sm + P::OFF_LINE),
                                           reinterpret_cast<long long*>(sm + P::OFF_SCAN), TU, CF_K, CHUNK_UNIT_F32, blockIdx.x == 0);
  const int parts = line.parts(p.parts), c = blockIdx.x;
  if (tid == 0) note_none(p, c);
  if (tid == 0 && c == 0) *p.queue = 0;
  if (c >= parts) return;
  const long long y0 = line.part_begin(parts, c), y1 = line.part_begin(parts, c + 1);
  const Patience patience{dead, p.status, p.wait_ns};
  int q_copies = 0, copies = 0, raw_copies = 0;  // that the copying warp has issued
  // (384 threads of 168 registers: 256 of 232 and 128 of 40)
  if (warp < CF_NT / 32) more_registers<232>();
  else fewer_registers<40>();
  if (warp < CF_NT / 32) {
    const int ty = tid >> 4, tx = tid & 15;
    uint32_t q_phase = 0, t_phase = 0;
    auto free_it = [&](uint32_t bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    segments(line, y0, y1, [&](const ChunkUnit& u, int f0, int f1, bool whole) {
      const int n = u.q.n, len = u.q.len, j0 = u.i * TU, rows = min(TU, n - j0) * p.G;
      const bool busy = 16 * warp < rows;  // whether this warp has rows
      if (tid == 0 && !whole) note_record(p, c, u, TU, f0, f1);
      float m[8], l[8];
      uint64_t o[8][2 * E];
      int see[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 8 * ty + i;
        m[i] = -INFINITY;
        l[i] = 0.f;
        see[i] = r < rows ? len - n + j0 + r / p.G + 1 : 0;
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) o[i][e] = 0;
      }
      if (f0 < f1) {
        if (!patience.wait(q_full, q_phase)) return false;
        q_phase ^= 1;
      }
      int odd = 0;
      for (int t = f0; t < f1; ++t) {
        const int t0 = t * CF_K;
        if (!patience.wait(k_full, t_phase)) return false;
        float z[8][4];
        int there = 0;  // of this thread's slots
        if (busy) {
          const unsigned h0 = held[2 * (t & 1)], h1 = held[2 * (t & 1) + 1];
          there = (h0 >> tx & 1) | (h0 >> (tx + 16) & 1) << 1 | (h1 >> tx & 1) << 2 | (h1 >> (tx + 16) & 1) << 3;
          products<D>(qs, ks, z);
        }
        free_it(k_empty);
        if (t + 1 == f1) free_it(q_empty);
        if (busy && chunk_light(p, u.b, u.q)) {
          float* keep = chunk_logits(p, u.b, u.h, u.q) + t0 + tx;
#pragma unroll 1
          for (int i = 0; 8 * ty + i < rows && i < 8; ++i)
            for (int j = 0; j < 4; ++j) {
              float x = 0.f;  // z[i][j], from registers
#pragma unroll
              for (int k = 0; k < 32; ++k) x = k == 4 * i + j ? z[k >> 2][k & 3] : x;
              keep[(size_t)(8 * ty + i) * p.T_pad + 16 * j] =
                  (there >> j & 1) && t0 + tx + 16 * j < len - n + j0 + (8 * ty + i) / p.G + 1 ? x * p.scale : -INFINITY;
            }
        }
        if (busy) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              z[i][j] = (there >> j & 1) && t0 + tx + 16 * j < see[i] ? z[i][j] * p.scale : -INFINITY;
              mx = fmaxf(mx, z[i][j]);
            }
#pragma unroll
            for (int s = 1; s < 16; s <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
            const float mn = fmaxf(m[i], mx), ms = mn == -INFINITY ? 0.f : mn;
            if (mn > m[i]) {
              const float a = exp2f(m[i] - ms);
              const uint64_t a2 = pair_of(a, a);
              l[i] *= a;
#pragma unroll
              for (int e = 0; e < 2 * E; ++e) o[i][e] = mul2(o[i][e], a2);
              m[i] = mn;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              z[i][j] = exp2f(z[i][j] - ms);
              ps[(8 * ty + i) * P::LP + tx + 16 * j] = z[i][j];
            }
            l[i] += (z[i][0] + z[i][1]) + (z[i][2] + z[i][3]);
          }
          __syncwarp();  // (P's rows are read by the lanes that wrote them)
        }
        if (!patience.wait(v_full, t_phase)) return false;
        t_phase ^= 1;
        odd |= *not_all_finite;
        if (busy) {
          const char* v0 = vs + (tx >> 3) * (CF_K * 128);
          uint64_t part[8][2 * E];  // of this tile
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 2 * E; ++e) part[i][e] = 0;
#pragma unroll 1
          for (int s8 = 0; s8 < CF_K; s8 += 8, v0 += 8 * 128) {
#pragma unroll
            for (int half = 0; half < 8; half += 4) {
              ulonglong2 v[4][E];
#pragma unroll
              for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int e = 0; e < E; ++e)
                  v[s][e] = *reinterpret_cast<const ulonglong2*>(v0 + 2 * e * (CF_K * 128) + (half + s) * 128 +
                                                                 (((half + s) ^ (tx & 7)) << 4));
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 w = *reinterpret_cast<const float4*>(ps + (8 * ty + i) * P::LP + s8 + half);
                const float ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                  const uint64_t w2 = pair_of(ws[s], ws[s]);
#pragma unroll
                  for (int e = 0; e < E; ++e) {
                    part[i][2 * e] = fma2(w2, v[s][e].x, part[i][2 * e]);
                    part[i][2 * e + 1] = fma2(w2, v[s][e].y, part[i][2 * e + 1]);
                  }
                }
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 2 * E; ++e) o[i][e] = add2(o[i][e], part[i][e]);
        }
        free_it(v_empty);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int s = 1; s < 16; s <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], s);
        const int r = 8 * ty + i;
        if (r >= rows) continue;
        const ChunkRow at(p, u, TU, r);
        float* rec = chunk_record(p, D, c, f0 > 0 ? 0 : 1);
        const float inv = !whole ? 1.f : l[i] > 0.f ? 1.f / l[i] : 0.f;
        float* to = whole ? static_cast<float*>(p.out) + at.out(p, D) : rec + (size_t)r * D;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float x[4];
          unpair(o[i][2 * e], x[0], x[1]);
          unpair(o[i][2 * e + 1], x[2], x[3]);
          store4<float>(to + 4 * tx + 64 * e, x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
        }
        if (tx == 0 && whole && p.weight) p.lse[at.lse(p)] = chunk_lse(m[i], l[i]);
        if (tx == 0 && !whole) {
          rec[(size_t)p.rows * D + r] = m[i];
          rec[(size_t)p.rows * (D + 1) + r] = l[i];
        }
      }
      if (odd) {  // (every thread the dims that it stored)
        const int s0 = max(partly_seen(u, TU).x, f0 * CF_K);
        for (int r = 8 * ty; r < min(rows, 8 * ty + 8); ++r) {
          float* to = whole ? static_cast<float*>(p.out) + ChunkRow(p, u, TU, r).out(p, D)
                            : chunk_record(p, D, c, f0 > 0 ? 0 : 1) + (size_t)r * D;
          for (int e = 0; e < E; ++e)
            add_not_finite<float>(p, u.b, u.h, s0, min(len - n + j0 + r / p.G + 1, f1 * CF_K), 4 * tx + 64 * e,
                                  4 * tx + 64 * e + 4, D, to);
        }
      }
      return true;
    });
  } else if (warp == CF_NT / 32) {
    // ------------------------------------------------ copies
    const int box = min(1 << p.log2_page, CF_K), per = CF_K / box;        // rows of a copy, copies of a slab
    const int none = (int)((long long)p.n_pages * p.Hkv << p.log2_page);  // a row behind the pool: zeros
    const int mine = lane / P::SLABS, slab = lane % P::SLABS;
    uint32_t q_phase = 1, t_phase = 1, raw_phase = 0;
    int n_tile = 0;
    fence_proxy_async_global();  // (a kernel before this one may have stored what is copied)
    segments(line, y0, y1, [&](const ChunkUnit& u, int f0, int f1, bool) {
      if (f0 == f1) return true;
      const int len = u.q.len;
      auto look_up = [&](int t) { return mine < per ? slot_row(p, u.b, u.h, t * CF_K + mine * box, len, true) : -1; };
      const int2 partly = partly_seen(u, TU);
      int next = look_up(f0);
      if (!patience.wait(q_empty, q_phase)) return false;
      q_phase ^= 1;
      if (lane == 0) mbar_arrive_expect_tx(q_full, P::SLABS * TU * p.G * 128);
      __syncwarp();
      ++q_copies;
      if (lane < P::SLABS) tma_3d(smem_u32(qs) + lane * CF_M * 128, &qmap, 32 * lane, u.h * p.G, u.q.first + u.i * TU, q_full);
      __syncwarp();
      for (int t = f0; t < f1; ++t) {
        const int row = next, behind = len - t * CF_K;  // slots before the end
        if (t + 1 < f1) next = look_up(t + 1);
        // which of the tile's boxes lie in the pool, and the mask of the slots that count
        const unsigned boxes = __ballot_sync(0xffffffffu, row >= 0 && slab == 0);
        unsigned h[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 2; ++i)
          h[i] = __ballot_sync(0xffffffffu, lane + 32 * i < behind && (boxes >> ((lane + 32 * i) / box * P::SLABS) & 1u));
        const bool drop = n_tile == p.drop_tile;  // (test hook: copies that never come)
        const int at = row >= 0 ? row : none;
        const uint32_t to = slab * CF_K * 128 + mine * box * 128;
        if (!patience.wait(k_empty, t_phase)) return false;
        if (lane == 0) {
          held[2 * (t & 1)] = h[0];
          held[2 * (t & 1) + 1] = h[1];
          mbar_arrive_expect_tx(k_full, P::K_BYTES);
        }
        __syncwarp();
        if (mine < per && !drop) tma_2d(smem_u32(ks) + to, &kmap, 32 * slab, at, k_full);
        __syncwarp();
        ++copies;
        if (!patience.wait(v_empty, t_phase)) return false;
        t_phase ^= 1;
        // Rows of V behind those that the unit sees have weights of 0 and may hold NaN: where
        // there are some in a page, they are cleared before V is passed on; elements that are not
        // finite, of slots that some of its rows do not see, too
        const bool tail = (t + 1) * CF_K > partly.x;
        if (lane == 0) *not_all_finite = 0;
        if (lane == 0) mbar_arrive_expect_tx(tail ? v_raw : v_full, P::K_BYTES);
        __syncwarp();
        if (mine < per && !drop) tma_2d(smem_u32(vs) + to, &vmap, 32 * slab, at, tail ? v_raw : v_full);
        __syncwarp();
        if (!tail) {
          ++copies;
        } else {
          ++raw_copies;
          if (!patience.wait(v_raw, raw_phase)) return false;
          raw_phase ^= 1;
          const int seen = min(CF_K, partly.y - t * CF_K), r0 = max(0, partly.x - t * CF_K);
          for (int i = lane; i < (CF_K - seen) * (D / 4); i += 32)
            *reinterpret_cast<float4*>(vs + swizzled(CF_K, seen + i / (D / 4), i % (D / 4))) = make_float4(0.f, 0.f, 0.f, 0.f);
          bool found = false;
#pragma unroll 4
          for (int i = lane; i < (seen - r0) * (D / 4); i += 32) {
            float4* at = reinterpret_cast<float4*>(vs + swizzled(CF_K, r0 + i / (D / 4), i % (D / 4)));
            float4 x = *at;
            if (not_finite(x.x) || not_finite(x.y) || not_finite(x.z) || not_finite(x.w)) {
              found = true;
              x.x = not_finite(x.x) ? 0.f : x.x;
              x.y = not_finite(x.y) ? 0.f : x.y;
              x.z = not_finite(x.z) ? 0.f : x.z;
              x.w = not_finite(x.w) ? 0.f : x.w;
              *at = x;
            }
          }
          if (__any_sync(0xffffffffu, found) && lane == 0) *not_all_finite = 1;
          fence_proxy_async();  // (before the next copy into them)
          __syncwarp();
          if (lane == 0) mbar_arrive(v_full);
          ++copies;
        }
        ++n_tile;
      }
      return true;
    });
  }
  // After a wait that ran out, no copy may land in memory of a block that is gone.
  __syncthreads();
  if (*dead && warp == CF_NT / 32) {
    // (the last copy into each place; V's, where it is a raw one, arrives there alone)
    const int ks_n = (copies + 1) / 2, vs_n = copies / 2;
    bool all = q_copies == 0 || mbar_wait_bounded(q_full, (q_copies - 1) & 1, 8 * p.wait_ns);
    all = (ks_n == 0 || mbar_wait_bounded(k_full, (ks_n - 1) & 1, 8 * p.wait_ns)) && all;
    all = (vs_n == 0 || mbar_wait_bounded(v_full, (vs_n - 1) & 1, 8 * p.wait_ns)) && all;
    all = (raw_copies == 0 || mbar_wait_bounded(v_raw, (raw_copies - 1) & 1, 8 * p.wait_ns)) && all;
    if (!all && lane == 0) atomicOr(p.status, 4);
  }
}

// weight_t += sum over the rows that see slot t of 2^(z_t - log2 of the row's sum): a unit
// is a tile of slots, the rows 128 at a time, added in their order; the next rows are on
// their way meanwhile.
template <int D>
__global__ void __launch_bounds__(CF_NT, 1) chunk_weight_f32_kernel(const __grid_constant__ ChunkParams p) {
  using P = CfPlan<D>;
  extern __shared__ __align__(16) char sm[];
  char* ks = sm;
  float* sums = reinterpret_cast<float*>(sm + P::W_SUM);
  int* rows_at = reinterpret_cast<int*>(sm + P::W_ROWS);
  int* before = reinterpret_cast<int*>(sm + P::W_LINE);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, TU = CF_M / p.G;
  paged_go();
  paged_wait();
  weight_line<CF_NT, CF_K>(p, before, reinterpret_cast<int3*>(sm + P::W_SCAN), TU);
  if (p.logits) weight_light<CF_NT>(p, before + 2 * (p.B + 1));
  __shared__ int ahead;
  for (int mine = blockIdx.x;;) {  // (the first unit is the block's own; the queue counts those behind)
    WeightUnit u;
    if (!weight_unit<CF_K>(p, before, mine, u)) return;
    if (tid == 0) ahead = gridDim.x + atomicAdd(p.queue, 1);
    const int from = u.from(0, TU), tiles = u.tiles(TU), a = u.q.len - u.q.n;
    auto fetch = [&](int i) {
      const int rows = min(TU, u.q.n - i * TU) * p.G;
      fetch_queries<D>(p, u.q.first + i * TU, u.h, rows, sm + P::W_Q + (i & 1) * P::Q_BYTES);
      if (tid < CF_M)  // (rows that there are not get nothing: 2^-inf)
        reinterpret_cast<float*>(sm + P::W_LSE)[(i & 1) * CF_M + tid] =
            tid < rows ? ld_cg(p.lse + ((size_t)u.h * p.n_tokens + u.q.first + i * TU) * p.G + tid) : INFINITY;
    };
    if (tid < CF_K) rows_at[tid] = slot_row(p, u.b, u.h, u.t0 + tid, u.q.len, false);
    __syncthreads();
    if (from < tiles) {
      fetch_slots<D>(p.k_pages, rows_at, ks);
      fetch(from);
    }
    float sum[4] = {};
    for (int i = from; i < tiles; ++i) {
      cp_async_wait<0>();
      __syncthreads();  // these rows are there, and those before them are read
      if (i + 1 < tiles) fetch(i + 1);
      const float* lse = reinterpret_cast<const float*>(sm + P::W_LSE) + (i & 1) * CF_M;
      float z[8][4];
      if (tid / 32 * 16 >= min(TU, u.q.n - i * TU) * p.G) continue;  // no rows of this warp
      products<D>(sm + P::W_Q + (i & 1) * P::Q_BYTES, ks, z);
      float part[4] = {};
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        // the last slot that this row sees (or the row that it is a copy of)
        const int see = a + i * TU + min((8 * ty + r) / p.G, TU - 1);
        const float x = lse[8 * ty + r];
#pragma unroll
        for (int j = 0; j < 4; ++j) part[j] += u.t0 + tx + 16 * j <= see ? exp2f(z[r][j] * p.scale - x) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += part[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sums[ty * P::LP + tx + 16 * j] = sum[j];
    __syncthreads();
    mine = ahead;
    if (tid < CF_K && rows_at[tid] >= 0) {
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) x += sums[i * P::LP + tid];
      if (x != 0.f) p.weight[((size_t)u.b * p.Hkv + u.h) * p.T_cap + u.t0 + tid] += x;
    }
    __syncthreads();  // (`ahead` and the sums are read)
  }
}

template <int D>
cudaError_t launch(const ChunkParams& p, cudaStream_t s) {
  using P = CfPlan<D>;
  static std::atomic<unsigned long long> allowed{0};  // devices that were told of the shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (!(allowed.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(chunk_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::bytes(PAGED_MAX_BATCH));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(chunk_weight_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               P::weight_bytes(PAGED_MAX_BATCH));
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_release);
  }
  const int TU = CF_M / p.G;
  CUtensorMap qm, km, vm;
  const cuuint64_t qd[3] = {D, (cuuint64_t)p.Hq, (cuuint64_t)p.n_tokens}, qst[2] = {D * 4, (cuuint64_t)p.Hq * D * 4};
  const cuuint32_t qb[3] = {32, (cuuint32_t)p.G, (cuuint32_t)TU};
  e = tensor_map(&qm, p.q, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, qd, qst, qb);
  const cuuint64_t kd[2] = {D, ((cuuint64_t)p.n_pages * p.Hkv) << p.log2_page}, kst[1] = {D * 4};
  const cuuint32_t kb[2] = {32, (cuuint32_t)std::min(1 << p.log2_page, CF_K)};
  if (e == cudaSuccess) e = tensor_map(&km, p.k_pages, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, kd, kst, kb);
  if (e == cudaSuccess) e = tensor_map(&vm, p.v_pages, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, kd, kst, kb);
  if (e == cudaSuccess) e = paged_behind(chunk_f32_kernel<D>, p.parts, CA_NT, P::bytes(p.B), 0, s, p, qm, km, vm);
  if (e == cudaSuccess) e = launch_chunk_join<float, D>(p, s);
  if (e == cudaSuccess && p.weight)
    e = paged_behind(chunk_weight_f32_kernel<D>, p.sms, CF_NT, P::weight_bytes(p.B), 0, s, p);
  return e;
}

}  // namespace

cudaError_t launch_chunk_f32(const ChunkParams& p, int head_dim, cudaStream_t s) {
  return head_dim == 128 ? launch<128>(p, s) : launch<64>(p, s);
}

}  // namespace fasa
