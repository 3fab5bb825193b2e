// Attention of chunks on CUDA cores.  A block takes a part of the line of units
// (fasa_chunk_index.h): 64 rows, the slots 64 at a time.
#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>

#include "fasa_cluster.cuh"
#include "fasa_chunk.cuh"

namespace fasa {
namespace {

constexpr int CF_NT = 256, CF_M = 64, CF_K = 64;

template <int D>
struct CfPlan {
  static constexpr int LD = D + 4;                 // (rows apart by four banks)
  static constexpr int OFF_KV = CF_M * LD * 4;
  static constexpr int OFF_P = OFF_KV + CF_K * LD * 4;
  static constexpr int LP = CF_K + 4;
  static constexpr int OFF_OK = OFF_P + CF_M * LP * 4;
  static constexpr int OFF_SCAN = OFF_OK + CF_K * 4;
  static constexpr int OFF_SEQ = OFF_SCAN + 64;
  static constexpr int bytes(int B) { return OFF_SEQ + (B + 1) * 8; }
};

// Slots t0 .. t0 + 63 of (b, h): rows of K or V in fp32, zeros for slots that do not
// count; ok[i]: whether slot t0 + i does.
template <typename T, int D>
__device__ __forceinline__ void load_slots(const ChunkParams& p, const void* pages, int b, int h, int t0, int len,
                                           float* to, int* ok) {
  constexpr int EPC = 16 / (int)sizeof(T), CH = D / EPC;
  for (int i = threadIdx.x; i < CF_K * CH; i += CF_NT) {
    const int r = i / CH, c = i % CH, t = t0 + r;
    long long row = -1;
    if (t < len)
      row = paged_row(p.page_table[(size_t)b * p.max_pages + (t >> p.log2_page)], p.n_pages, p.Hkv, h, p.log2_page, t);
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (row >= 0) w = *reinterpret_cast<const uint4*>(static_cast<const T*>(pages) + row * D + c * EPC);
    float* x = to + r * CfPlan<D>::LD + c * EPC;
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = bf16_lo(u[e]);
        x[2 * e + 1] = bf16_hi(u[e]);
      }
    } else {
      *reinterpret_cast<uint4*>(x) = w;
    }
    if (c == 0 && ok) {
      ok[r] = row >= 0;
      if (t < len && row < 0) atomicOr(p.status, 1);
    }
  }
}

// Rows [r0, r0 + 64) of a sequence's tokens from j0 on, head group h.
template <typename T, int D>
__device__ __forceinline__ void load_queries(const ChunkParams& p, int first, int j0, int n, int h, float* to) {
  constexpr int EPC = 16 / (int)sizeof(T), CH = D / EPC;
  for (int i = threadIdx.x; i < CF_M * CH; i += CF_NT) {
    const int r = i / CH, c = i % CH, j = j0 + r / p.G;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (r < CF_M / p.G * p.G && j < n)
      w = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) +
                                          ((size_t)(first + j) * p.Hq + h * p.G + r % p.G) * D + c * EPC);
    float* x = to + r * CfPlan<D>::LD + c * EPC;
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = bf16_lo(u[e]);
        x[2 * e + 1] = bf16_hi(u[e]);
      }
    } else {
      *reinterpret_cast<uint4*>(x) = w;
    }
  }
}

// z[i][j]: row 4 ty + i, slot tx + 16 j.
template <int D>
__device__ __forceinline__ void products(const float* q, const float* k, float (&z)[4][4]) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i >> 2][i & 3] = 0.f;
#pragma unroll 4
  for (int c = 0; c < D / 4; ++c) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = *reinterpret_cast<const float4*>(q + (4 * ty + i) * CfPlan<D>::LD + 4 * c);
      b[i] = *reinterpret_cast<const float4*>(k + (tx + 16 * i) * CfPlan<D>::LD + 4 * c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        z[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, z[i][j]))));
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(CF_NT) chunk_simt_kernel(const __grid_constant__ ChunkParams p) {
  using P = CfPlan<D>;
  constexpr int E = D / 16;
  extern __shared__ __align__(16) char sm[];
  float* qs = reinterpret_cast<float*>(sm);
  float* kv = reinterpret_cast<float*>(sm + P::OFF_KV);
  float* ps = reinterpret_cast<float*>(sm + P::OFF_P);
  int* ok = reinterpret_cast<int*>(sm + P::OFF_OK);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, TU = CF_M / p.G;
  paged_wait();
  paged_go();
  const ChunkLine line = chunk_line<CF_NT>(p, reinterpret_cast<long long*>(sm + P::OFF_SEQ),
                                           reinterpret_cast<long long*>(sm + P::OFF_SCAN), TU, CF_K, blockIdx.x == 0);
  const int parts = line.parts(p.parts), c = blockIdx.x;
  if (tid == 0) note_none(p, c);
  if (c >= parts) return;
  const long long y0 = line.part_begin(parts, c), y1 = line.part_begin(parts, c + 1);
  ChunkUnit u;
  for (u.find(line, y0); u.begin < y1;) {
    const int f0 = u.before(line, y0), f1 = u.before(line, y1), n = u.q.n, len = u.q.len;
    const bool whole = f0 == 0 && f1 == u.tiles && u.begin >= y0;
    if (f0 < f1 || whole) {
      if (tid == 0 && !whole) note_record(p, c, u, TU, f0, f1);
      const int first = u.q.first, j0 = u.i * TU, rows = min(TU, n - j0) * p.G;
      __syncthreads();
      load_queries<T, D>(p, first, j0, n, u.h, qs);
      float m[4], l[4], o[4][E];
      int see[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        m[i] = -INFINITY;
        l[i] = 0.f;
        see[i] = r < rows ? len - n + j0 + r / p.G + 1 : 0;
#pragma unroll
        for (int e = 0; e < E; ++e) o[i][e] = 0.f;
      }
      for (int t = f0; t < f1; ++t) {
        const int t0 = t * CF_K;
        __syncthreads();
        load_slots<T, D>(p, p.k_pages, u.b, u.h, t0, len, kv, ok);
        __syncthreads();
        float z[4][4];
        products<D>(qs, kv, z);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float mx = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int s = tx + 16 * j;
            z[i][j] = ok[s] && t0 + s < see[i] ? z[i][j] * p.scale : -INFINITY;
            mx = fmaxf(mx, z[i][j]);
          }
#pragma unroll
          for (int s = 1; s < 16; s <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
          const float mn = fmaxf(m[i], mx), ms = mn == -INFINITY ? 0.f : mn, a = exp2f(m[i] - ms);
          m[i] = mn;
          l[i] *= a;
#pragma unroll
          for (int e = 0; e < E; ++e) o[i][e] *= a;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float w = exp2f(z[i][j] - ms);
            l[i] += w;
            ps[(4 * ty + i) * P::LP + tx + 16 * j] = w;
          }
        }
        __syncthreads();
        load_slots<T, D>(p, p.v_pages, u.b, u.h, t0, len, kv, nullptr);
        __syncthreads();
        for (int s = 0; s < CF_K; ++s) {
          float v[E];
#pragma unroll
          for (int e = 0; e < E; e += 4) {
            const float4 x = *reinterpret_cast<const float4*>(kv + s * P::LD + 4 * tx + 16 * e);
            v[e] = x.x;
            v[e + 1] = x.y;
            v[e + 2] = x.z;
            v[e + 3] = x.w;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float w = ps[(4 * ty + i) * P::LP + s];
#pragma unroll
            for (int e = 0; e < E; ++e) o[i][e] = fmaf(w, v[e], o[i][e]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int s = 1; s < 16; s <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], s);
        const int r = 4 * ty + i;
        if (r >= rows) continue;
        const ChunkRow at(p, u, TU, r);
        if (whole) {
          const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
          T* to = static_cast<T*>(p.out) + at.out(p, D);
#pragma unroll
          for (int e = 0; e < E; e += 4)
            store4<T>(to + 4 * tx + 16 * e, o[i][e] * inv, o[i][e + 1] * inv, o[i][e + 2] * inv, o[i][e + 3] * inv);
          if (p.weight && tx == 0) p.lse[at.lse(p)] = chunk_lse(m[i], l[i]);
        } else {
          float* rec = chunk_record(p, D, c, f0 > 0 ? 0 : 1);
#pragma unroll
          for (int e = 0; e < E; e += 4)
            store4<float>(rec + (size_t)r * D + 4 * tx + 16 * e, o[i][e], o[i][e + 1], o[i][e + 2], o[i][e + 3]);
          if (tx == 0) {
            rec[(size_t)p.rows * D + r] = m[i];
            rec[(size_t)p.rows * (D + 1) + r] = l[i];
          }
        }
      }
    }
    if (u.begin + u.cost >= y1) break;
    u.next(line);
  }
}

// weight_t += sum over the rows that see slot t of 2^(z_t - log2 of the row's sum): one
// block a tile of slots, the rows 64 at a time, added in their order.
template <typename T, int D>
__global__ void __launch_bounds__(CF_NT) chunk_simt_weight_kernel(const __grid_constant__ ChunkParams p) {
  using P = CfPlan<D>;
  extern __shared__ __align__(16) char sm[];
  float* qs = reinterpret_cast<float*>(sm);
  float* ks = reinterpret_cast<float*>(sm + P::OFF_KV);
  float* sums = reinterpret_cast<float*>(sm + P::OFF_P);
  int* ok = reinterpret_cast<int*>(sm + P::OFF_OK);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, TU = CF_M / p.G;
  paged_go();
  paged_wait();
  const int tiles = (p.T_cap + CF_K - 1) / CF_K;
  const long long units = (long long)p.B * tiles * p.Hkv;
  for (long long w = blockIdx.x; w < units; w += gridDim.x) {
    const int b = (int)(w / ((long long)tiles * p.Hkv)), rem = (int)(w - (long long)b * tiles * p.Hkv);
    const int t = rem / p.Hkv, h = rem % p.Hkv, t0 = t * CF_K;
    const int len = min(max(p.seq_lens[b], 0), p.T_cap);
    if (t0 >= len) continue;
    int first = b, n = 1;
    if (p.cu_new) {
      first = p.cu_new[b];
      const int end = p.cu_new[b + 1];
      n = 0 <= first && first <= end && end <= p.n_tokens ? end - first : 0;
    }
    const int a = len - n, from = max(0, t0 - a) / TU;  // the first tile of rows that sees the slots
    __syncthreads();
    load_slots<T, D>(p, p.k_pages, b, h, t0, len, ks, ok);
    float sum[4] = {};
    for (int i0 = from; i0 * TU < n; ++i0) {
      const int j0 = i0 * TU;
      __syncthreads();
      load_queries<T, D>(p, first, j0, n, h, qs);
      __syncthreads();
      float z[4][4];
      products<D>(qs, ks, z);
      float part[4] = {};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i, jr = j0 + r / p.G;
        if (r < TU * p.G && jr < n) {
          const float lse = ld_cg(p.lse + ((size_t)h * p.n_tokens + first + jr) * p.G + r % p.G);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (t0 + tx + 16 * j <= a + jr) part[j] += exp2f(z[i][j] * p.scale - lse);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += part[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) sums[ty * P::LP + tx + 16 * j] = sum[j];
    __syncthreads();
    if (tid < CF_K && ok[tid]) {
      float x = 0.f;
      for (int i = 0; i < CF_NT / 16; ++i) x += sums[i * P::LP + tid];
      if (x != 0.f) p.weight[((size_t)b * p.Hkv + h) * p.T_cap + t0 + tid] += x;
    }
  }
}

template <typename T, int D>
cudaError_t launch(const ChunkParams& p, cudaStream_t s) {
  using P = CfPlan<D>;
  static std::atomic<unsigned long long> allowed{0};  // devices that were told of the shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (!(allowed.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(chunk_simt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::bytes(PAGED_MAX_BATCH));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(chunk_simt_weight_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::OFF_SCAN);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_release);
  }
  e = paged_behind(chunk_simt_kernel<T, D>, p.parts, CF_NT, P::bytes(p.B), 0, s, p);
  if (e == cudaSuccess) e = launch_chunk_join<T, D>(p, s);
  if (e == cudaSuccess && p.weight) {
    const long long units = (long long)p.B * p.Hkv * ((p.T_cap + CF_K - 1) / CF_K);
    e = paged_behind(chunk_simt_weight_kernel<T, D>, (unsigned)(units < 4096 ? units : 4096), CF_NT, P::OFF_SCAN, 0, s, p);
  }
  return e;
}

}  // namespace

cudaError_t launch_chunk_f32(const ChunkParams& p, int head_dim, cudaStream_t s) {
  return head_dim == 128 ? launch<float, 128>(p, s) : launch<float, 64>(p, s);
}

}  // namespace fasa
