// Attention of chunks in fp32 on CUDA cores.  A block takes a part of the line of units
// (fasa_chunk_index.h): up to 128 rows (new tokens times the heads of their group), the
// slots 64 at a time.
//
// A thread has 8 rows and 4 slots of Z = Q K^T and 8 rows and D / 16 dims of O, its products
// two at a time (fma.f32x2: the instruction alone would fill the issue slots that the
// operands' loads need too).  K of the next tile is on its way while P V is worked out, V
// while Q K^T is.  Bound by the products: 1500 tokens of heads of 128 dims run at 60% of
// the FMA rate.
#include <stdint.h>

#include <atomic>

#include "fasa_cluster.cuh"
#include "fasa_chunk.cuh"
#include "fasa_tcgen05.cuh"

namespace fasa {
namespace {

constexpr int CF_NT = 256, CF_M = 128, CF_K = 64;
constexpr int CF_UNIT = 48;  // what a unit costs beside its tiles, in slots

template <int D>
struct CfPlan {
  static constexpr int LD = D + 4;   // floats of a row (rows apart by four banks)
  static constexpr int LP = CF_K + 4;
  static constexpr int Q_BYTES = CF_M * LD * 4, K_BYTES = CF_K * LD * 4;
  // attention: Q, K, V, P, where the slots' rows lie (two tiles), the line
  static constexpr int OFF_K = Q_BYTES, OFF_V = OFF_K + K_BYTES, OFF_P = OFF_V + K_BYTES;
  static constexpr int OFF_ROWS = OFF_P + CF_M * LP * 4;
  static constexpr int OFF_SCAN = OFF_ROWS + 2 * CF_K * 4;
  static constexpr int OFF_LINE = OFF_SCAN + CF_NT / 32 * 8;
  static constexpr int bytes(int B) { return OFF_LINE + (B + 1) * 8; }
  // weights: K, Q and its rows' log-sums twice, sums
  static constexpr int W_Q = K_BYTES, W_LSE = W_Q + 2 * Q_BYTES, W_SUM = W_LSE + 2 * CF_M * 4;
  static constexpr int W_ROWS = W_SUM + 16 * LP * 4, W_SCAN = W_ROWS + CF_K * 4, W_LINE = W_SCAN + CF_NT / 32 * 8;
  static constexpr int weight_bytes(int B) { return W_LINE + (2 * B + 2) * 4; }
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

// 64 rows of K or V, zeros for those that do not count (what such memory holds may be NaN).
template <int D>
__device__ __forceinline__ void fetch_slots(const void* pages, const int* rows, float* to) {
  constexpr int CH = D / 4;
#pragma unroll
  for (int i = threadIdx.x; i < CF_K * CH; i += CF_NT) {
    const int r = i / CH, c = i % CH, row = rows[r];
    cp_async16_zfill(smem_u32(to + r * CfPlan<D>::LD + 4 * c),
                     static_cast<const float*>(pages) + (size_t)max(row, 0) * D + 4 * c, row >= 0 ? 16u : 0u);
  }
  cp_async_commit();
}

// Rows of a unit's queries: `count` of them from token `token` on, head group h; zeros behind.
template <int D>
__device__ __forceinline__ void fetch_queries(const ChunkParams& p, int token, int h, int count, float* to) {
  constexpr int CH = D / 4;
#pragma unroll 4
  for (int i = threadIdx.x; i < CF_M * CH; i += CF_NT) {
    const int r = i / CH, c = i % CH, j = r / p.G;
    const bool live = r < count;
    const size_t from = ((size_t)(token + (live ? j : 0)) * p.Hq + h * p.G + (live ? r - j * p.G : 0)) * D + 4 * c;
    cp_async16_zfill(smem_u32(to + r * CfPlan<D>::LD + 4 * c), static_cast<const float*>(p.q) + from, live ? 16u : 0u);
  }
  cp_async_commit();
}

// z[i][j]: row 8 ty + i, slot tx + 16 j.  The even and the odd dims add up apart.
template <int D>
__device__ __forceinline__ void products(const float* q, const float* k, float (&z)[8][4]) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  uint64_t acc[8][4];
#pragma unroll
  for (int i = 0; i < 32; ++i) acc[i >> 2][i & 3] = 0;
#pragma unroll 2
  for (int c = 0; c < D / 4; ++c) {
    ulonglong2 b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const ulonglong2*>(k + (tx + 16 * j) * CfPlan<D>::LD + 4 * c);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(q + (8 * ty + i) * CfPlan<D>::LD + 4 * c);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fma2(a.y, b[j].y, fma2(a.x, b[j].x, acc[i][j]));
    }
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    float x, y;
    unpair(acc[i >> 2][i & 3], x, y);
    z[i >> 2][i & 3] = x + y;
  }
}

template <int D>
__global__ void __launch_bounds__(CF_NT, 1) chunk_f32_kernel(const __grid_constant__ ChunkParams p) {
  using P = CfPlan<D>;
  constexpr int E = D / 64;  // groups of 4 dims of a thread: 4 tx + 64 e ..
  extern __shared__ __align__(16) char sm[];
  float* qs = reinterpret_cast<float*>(sm);
  float* ks = reinterpret_cast<float*>(sm + P::OFF_K);
  float* vs = reinterpret_cast<float*>(sm + P::OFF_V);
  float* ps = reinterpret_cast<float*>(sm + P::OFF_P);
  int* rows_at = reinterpret_cast<int*>(sm + P::OFF_ROWS);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, TU = CF_M / p.G;
  paged_wait();
  paged_go();
  const ChunkLine line = chunk_line<CF_NT>(p, reinterpret_cast<long long*>(sm + P::OFF_LINE),
                                           reinterpret_cast<long long*>(sm + P::OFF_SCAN), TU, CF_K, CF_UNIT, blockIdx.x == 0);
  const int parts = line.parts(p.parts), c = blockIdx.x;
  if (tid == 0) note_none(p, c);
  if (tid == 0 && c == 0) *p.queue = 0;
  if (c >= parts) return;
  const long long y0 = line.part_begin(parts, c), y1 = line.part_begin(parts, c + 1);
  ChunkUnit u;
  for (u.find(line, y0); u.begin < y1; u.next(line)) {
    const int f0 = u.before(line, y0), f1 = u.before(line, y1), n = u.q.n, len = u.q.len;
    const bool whole = f0 == 0 && f1 == u.tiles && u.begin >= y0;
    if (f0 < f1 || whole) {
      if (tid == 0 && !whole) note_record(p, c, u, TU, f0, f1);
      const int j0 = u.i * TU, rows = min(TU, n - j0) * p.G;
      __syncthreads();
      fetch_queries<D>(p, u.q.first + j0, u.h, rows, qs);
      int next = -1;  // where a slot of the tile after lies
      if (f0 < f1) {
        if (tid < CF_K) rows_at[(f0 & 1) * CF_K + tid] = slot_row(p, u.b, u.h, f0 * CF_K + tid, len, true);
        if (tid < CF_K && f0 + 1 < f1) next = slot_row(p, u.b, u.h, (f0 + 1) * CF_K + tid, len, true);
        __syncthreads();
        fetch_slots<D>(p.k_pages, rows_at + (f0 & 1) * CF_K, ks);
        fetch_slots<D>(p.v_pages, rows_at + (f0 & 1) * CF_K, vs);
      }
      const bool busy = tid / 32 * 16 < rows;  // whether this warp has rows
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
      for (int t = f0; t < f1; ++t) {
        const int t0 = t * CF_K, *here = rows_at + (t & 1) * CF_K;
        const bool more = t + 1 < f1;
        cp_async_wait<1>();  // (V may be under way)
        if (tid < CF_K) rows_at[(t + 1 & 1) * CF_K + tid] = next;
        __syncthreads();
        if (tid < CF_K && t + 2 < f1) next = slot_row(p, u.b, u.h, t0 + 2 * CF_K + tid, len, true);
        if (busy) {
          float z[8][4];
          products<D>(qs, ks, z);
          int there = 0;  // of this thread's slots
#pragma unroll
          for (int j = 0; j < 4; ++j) there |= (here[tx + 16 * j] >= 0) << j;
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
              const float w = exp2f(z[i][j] - ms);
              l[i] += w;
              ps[(8 * ty + i) * P::LP + tx + 16 * j] = w;
            }
          }
        }
        cp_async_wait<0>();
        __syncthreads();  // K is read, P and V are there
        if (more) fetch_slots<D>(p.k_pages, rows_at + (t + 1 & 1) * CF_K, ks);
        if (busy) {
#pragma unroll 2
          for (int s4 = 0; s4 < CF_K; s4 += 4) {
            ulonglong2 v[4][E];
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
              for (int e = 0; e < E; ++e) v[s][e] = *reinterpret_cast<const ulonglong2*>(vs + (s4 + s) * P::LD + 4 * tx + 64 * e);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 w = *reinterpret_cast<const float4*>(ps + (8 * ty + i) * P::LP + s4);
              const float ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int s = 0; s < 4; ++s) {
                const uint64_t w2 = pair_of(ws[s], ws[s]);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                  o[i][2 * e] = fma2(w2, v[s][e].x, o[i][2 * e]);
                  o[i][2 * e + 1] = fma2(w2, v[s][e].y, o[i][2 * e + 1]);
                }
              }
            }
          }
        }
        __syncthreads();  // V and P are read
        if (more) fetch_slots<D>(p.v_pages, rows_at + (t + 1 & 1) * CF_K, vs);
      }
      cp_async_wait<0>();  // (of a unit without tiles: its Q)
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
    }
    if (u.begin + u.cost >= y1) break;
  }
}

// weight_t += sum over the rows that see slot t of 2^(z_t - log2 of the row's sum): a unit
// is a tile of slots, the rows 128 at a time, added in their order; the next rows are on
// their way meanwhile.
template <int D>
__global__ void __launch_bounds__(CF_NT, 1) chunk_weight_f32_kernel(const __grid_constant__ ChunkParams p) {
  using P = CfPlan<D>;
  extern __shared__ __align__(16) char sm[];
  float* ks = reinterpret_cast<float*>(sm);
  float* sums = reinterpret_cast<float*>(sm + P::W_SUM);
  int* rows_at = reinterpret_cast<int*>(sm + P::W_ROWS);
  int* before = reinterpret_cast<int*>(sm + P::W_LINE);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, TU = CF_M / p.G;
  paged_go();
  paged_wait();
  weight_line<CF_NT, CF_K>(p, before, reinterpret_cast<int2*>(sm + P::W_SCAN), TU);
  __shared__ int ahead;
  for (int mine = blockIdx.x;;) {  // (the first unit is the block's own; the queue counts those behind)
    WeightUnit u;
    if (!weight_unit<CF_K>(p, before, mine, u)) return;
    if (tid == 0) ahead = gridDim.x + atomicAdd(p.queue, 1);
    const int from = u.from(0, TU), tiles = u.tiles(TU), a = u.q.len - u.q.n;
    auto fetch = [&](int i) {
      const int rows = min(TU, u.q.n - i * TU) * p.G;
      fetch_queries<D>(p, u.q.first + i * TU, u.h, rows, reinterpret_cast<float*>(sm + P::W_Q + (i & 1) * P::Q_BYTES));
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
      products<D>(reinterpret_cast<const float*>(sm + P::W_Q + (i & 1) * P::Q_BYTES), ks, z);
      float part[4] = {};
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int see = a + i * TU + (8 * ty + r) / p.G;  // the last slot that this row sees
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
  e = paged_behind(chunk_f32_kernel<D>, p.parts, CF_NT, P::bytes(p.B), 0, s, p);
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
