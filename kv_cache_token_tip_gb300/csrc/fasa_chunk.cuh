// What the kernels of the attention of chunks share: the line of units in shared
// memory, and the join of units that were cut.
//
// For a row (a new token and a query head) with z_t = log2(e) q . K_t / sqrt(d) over the
// slots that the token sees: m = max z_t, l = sum 2^(z_t - m), o = sum 2^(z_t - m) V_t,
// out = o / l.  Two parts (m, l, o), (m', l', o') of a row join as M = max(m, m'),
// l 2^(m - M) + l' 2^(m' - M), and o alike.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "fasa_ptx.cuh"
#include "fasa_serve.h"

namespace fasa {

// The sequences' words.  Every thread of the block calls it; ends with a barrier.
// scan: NT / 32 words.  Lengths and rows are read past L1, since the join reads them
// ahead of its wait.
template <int NT>
__device__ void chunk_line(const ChunkParams& p, ChunkSeq* s, long long* scan, int T, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (p.B + NT - 1) / NT, b0 = min(p.B, tid * run), b1 = min(p.B, b0 + run);
  bool bad = false;
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    int len = ld_cg(p.seq_lens + b);
    bad = bad || len < 0 || len > p.T_cap;
    len = min(max(len, 0), p.T_cap);
    int n = 1;
    if (p.cu_new) {
      const int x0 = ld_cg(p.cu_new + b), x1 = ld_cg(p.cu_new + b + 1);
      const bool ok = 0 <= x0 && x0 <= x1 && x1 <= p.n_tokens;
      bad = bad || !ok || (b == 0 && x0 != 0);
      n = ok ? x1 - x0 : 0;
    }
    s[b].before = sum;
    s[b].n = n;
    s[b].len = len;
    sum += ChunkLine::cost_of(n, len, T);
  }
  if (report && bad) atomicOr(p.status, 1);
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  long long before = incl - sum;
#pragma unroll
  for (int v = 0; v < NT / 32; ++v) before += v < warp ? scan[v] : 0;
  for (int b = b0; b < b1; ++b) s[b].before += before;
  if (tid == NT - 1) {
    s[p.B].before = before + sum;
    s[p.B].n = s[p.B].len = 0;
  }
  __syncthreads();
}

__device__ __forceinline__ int first_row(const ChunkParams& p, int b) { return p.cu_new ? p.cu_new[b] : b; }

// Place of row r of unit u in `out` and in the log-sums: its token and head.
struct ChunkRow {
  int token, head;  // of the call's rows; of the Hq heads
  __device__ ChunkRow(const ChunkParams& p, const ChunkUnit& u, int first, int T, int r)
      : token(first + u.i * T + r / p.G), head(u.h * p.G + r % p.G) {}
  __device__ size_t out(const ChunkParams& p, int D) const { return ((size_t)token * p.Hq + head) * D; }
  __device__ size_t lse(const ChunkParams& p) const {
    return ((size_t)(head / p.G) * p.n_tokens + token) * p.G + head % p.G;
  }
};

__device__ __forceinline__ float chunk_lse(float m, float l) { return l > 0.f ? m + log2f(l) : INFINITY; }

template <typename T>
__device__ __forceinline__ void store4(T* to, float a, float b, float c, float d) {
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16(a, b), pack_bf16(c, d));
  else
    *reinterpret_cast<float4*>(to) = make_float4(a, b, c, d);
}

// Record of part c: slot 0 of a unit that began before it, slot 1 of one that goes on.
__device__ __forceinline__ float* chunk_record(const ChunkParams& p, int D, int c, int slot) {
  return p.records + (size_t)(2 * c + slot) * ((size_t)p.rows * (D + 2));
}

// The units that were cut: block x takes the cut before part x + 1 if it is the first of
// its unit, its warps the rows.  The parts of a row are added in part order.
constexpr int CJ_NT = 256;
constexpr int CJ_ROWS = 32;  // rows of a block
template <typename T, int D>
__global__ void __launch_bounds__(CJ_NT) chunk_join_kernel(const __grid_constant__ ChunkParams p, int T_unit, int KT) {
  extern __shared__ __align__(16) ChunkSeq seqs[];
  __shared__ long long scan[CJ_NT / 32];
  __shared__ int before[2 * CHUNK_MAX_SMS + 2];
  chunk_line<CJ_NT>(p, seqs, scan, T_unit, false);
  const ChunkLine line{seqs, p.B, p.Hkv, T_unit, KT};
  const int parts = line.parts(p.parts), c = blockIdx.x + 1;
  paged_go();
  paged_wait();
  if (c >= parts) return;
  ChunkUnit u;
  u.find(line, line.part_begin(parts, c));
  // tiles of the unit that lie before the cuts c - 1, c, c + 1, ..
  for (int k = threadIdx.x; k <= parts - c + 1; k += CJ_NT) before[k] = u.before(line, line.part_begin(parts, c - 1 + k));
  __syncthreads();
  if (before[0] > 0 || before[1] == 0 || before[1] == u.tiles) return;
  const int n = min(T_unit, seqs[u.b].n - u.i * T_unit) * p.G, first = first_row(p, u.b);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int E = D / 32, U = 4;  // U: parts that a lane has on the way
  for (int r = blockIdx.y * CJ_ROWS + warp; r < min(n, (int)(blockIdx.y + 1) * CJ_ROWS); r += CJ_NT / 32) {
    float M = -INFINITY, L = 0.f, o[E] = {};
    for (int k0 = 0; before[k0] < u.tiles; k0 += U) {
      float x[U][E], m[U], l[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int k = min(k0 + i, parts - c);
        // (a part without a tile of the unit left no record)
        const bool any = k == k0 + i && before[k] < before[k + 1];
        const float* rec = chunk_record(p, D, c - 1 + k, k == 0);
        m[i] = any ? ld_cg(rec + (size_t)p.rows * D + r) : -INFINITY;
        l[i] = any ? ld_cg(rec + (size_t)p.rows * (D + 1) + r) : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x[i][e] = any ? ld_cg(rec + (size_t)r * D + 32 * e + lane) : 0.f;
      }
      float X = M;
#pragma unroll
      for (int i = 0; i < U; ++i) X = fmaxf(X, m[i]);
      const float Xs = X == -INFINITY ? 0.f : X, f = exp2f(M - Xs);
      M = X;
      L *= f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const float g = exp2f(m[i] - Xs);
        L += l[i] * g;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += x[i][e] * g;
      }
      if (k0 + U > parts - c) break;
    }
    const ChunkRow at(p, u, first, T_unit, r);
    const float inv = L > 0.f ? 1.f / L : 0.f;
    T* to = static_cast<T*>(p.out) + at.out(p, D);
#pragma unroll
    for (int e = 0; e < E; ++e) to[32 * e + lane] = from_f32<T>(o[e] * inv);
    if (p.weight && lane == 0) p.lse[at.lse(p)] = chunk_lse(M, L);
  }
}

template <typename T, int D>
cudaError_t launch_chunk_join(const ChunkParams& p, int T_unit, int KT, cudaStream_t s) {
  if (p.parts < 2) return cudaSuccess;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.parts - 1, (p.rows + CJ_ROWS - 1) / CJ_ROWS);
  cfg.blockDim = dim3(CJ_NT);
  cfg.dynamicSmemBytes = (p.B + 1) * sizeof(ChunkSeq);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_join_kernel<T, D>, p, T_unit, KT);
}

}  // namespace fasa
