// Attention of one new token per sequence over the paged cache, split over
// the cache's length and joined, and the accumulated attention weights.
//
// For a unit (sequence b, KV head h) with the rotated query q_g of each of its
// G heads and z_gt = log2(e) q_g . K_t / sqrt(d):
//   m_g = max_t z_gt,  l_g = sum_t 2^(z_gt - m_g),  o_g = sum_t 2^(z_gt - m_g) V_t,
//   out_g = o_g / l_g,  weight_t += sum_g 2^(z_gt - m_g - log2 l_g).
// Two parts (m, l, o), (m', l', o') of a unit join as M = max(m, m'),
// l 2^(m - M) + l' 2^(m' - M), and o alike.
//
// attend: each CTA takes one part of the line of all token groups
// (fasa_paged_index.h), unit by unit; its warps take groups in turn, each with
// a running (m, l, o) of its own, joined at the unit's end in the CTA.  A unit
// the CTA holds whole is finished there; otherwise its record goes to the
// workspace.  join: the records of a unit that was cut, in part order; and
// with weights, a second pass over the logits the first one left.
#include <cuda_bf16.h>
#include <stdint.h>

#include "fasa_cluster.cuh"
#include "fasa_internal.h"
#include "fasa_paged.h"
#include "fasa_ptx.cuh"

namespace fasa {
namespace {

constexpr int AT_NT = 256;
constexpr int AT_NW = AT_NT / 32;

__device__ __forceinline__ int clamped_len(const PagedCommon& p, int b) {
  return min(max(p.seq_lens[b], 0), p.T_cap);
}

// pre[b] = groups of the sequences before b, b = 0 .. B.  Every thread calls
// it; ends with a barrier.
template <int NT>
__device__ void group_prefix(const PagedCommon& p, int* pre, int* scan, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int base = 0;
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    const int b = b0 + tid;
    int n = 0;
    if (b < p.B) {
      const int len = p.seq_lens[b];
      if (report && (len < 0 || len > p.T_cap)) atomicOr(p.status, 1);
      n = paged_groups(min(max(len, 0), p.T_cap));
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int before = base, tot = 0;
    for (int w = 0; w < NT / 32; ++w) {
      before += w < warp ? scan[w] : 0;
      tot += scan[w];
    }
    if (b < p.B) pre[b + 1] = before + incl;
    base += tot;
    __syncthreads();
  }
  if (tid == 0) pre[0] = 0;
  __syncthreads();
}

// The sequence whose units hold position x of the line.
__device__ __forceinline__ int sequence_of(const int* pre, int B, int Hkv, int x) {
  int lo = 0, hi = B;  // Hkv * pre[lo] <= x < Hkv * pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] * Hkv <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Walks the units that [x, end) of the line touches.
struct Segments {
  const int* pre;
  int Hkv, end;
  int x, b, h;           // where the next segment begins
  int unit_begin, unit_end;
  __device__ void start(const int* pre_, int B, int Hkv_, int x_, int end_) {
    pre = pre_;
    Hkv = Hkv_;
    x = x_;
    end = end_;
    b = x < end ? sequence_of(pre, B, Hkv, x) : 0;
    const int n = pre[b + 1] - pre[b];
    h = n ? (x - pre[b] * Hkv) / n : 0;
  }
  // The segment at x: its unit (b, h) and where the unit lies; false at the end.
  __device__ bool at() {
    if (x >= end) return false;
    while (pre[b + 1] == pre[b]) ++b;
    const int n = pre[b + 1] - pre[b];
    unit_begin = pre[b] * Hkv + h * n;
    unit_end = unit_begin + n;
    return true;
  }
  __device__ int seg_end() const { return min(unit_end, end); }
  __device__ void next() {
    x = seg_end();
    if (x == unit_end && ++h == Hkv) {
      h = 0;
      ++b;
    }
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(AT_NT) paged_attend_kernel(const __grid_constant__ PagedAttendParams p) {
  constexpr int E = D / 32;
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.G;
  float* qs = sm;                      // [G][D]
  float* mrg = qs + G_MAX * D;         // [AT_NW][G][D]
  float* mml = mrg + AT_NW * G_MAX * D;  // [AT_NW][G][2]
  int* scan = reinterpret_cast<int*>(mml + AT_NW * G_MAX * 2);
  int* pre = scan + 32;
  group_prefix<AT_NT>(p, pre, scan, blockIdx.x == 0);
  const int total = pre[p.B] * p.Hkv;
  const int parts = paged_parts(total, p.grid);
  const int c = blockIdx.x;
  // sequences without a token: zeros
  for (int b = c; b < p.B; b += p.grid)
    if (pre[b] == pre[b + 1])
      for (int i = tid; i < p.Hq * D; i += AT_NT) p.out[(size_t)b * p.Hq * D + i] = 0.f;
  if (tid == 0) p.joins[c] = make_int2(-1, 0);
  if (c >= parts) return;
  const int r0 = paged_part_begin(total, parts, c), r1 = paged_part_begin(total, parts, c + 1);
  Segments sg;
  sg.start(pre, p.B, p.Hkv, r0, r1);
  while (sg.at()) {
    const int b = sg.b, h = sg.h, unit = b * p.Hkv + h;
    const int len = clamped_len(p, b);
    __syncthreads();
    for (int i = tid; i < G * (D / 2); i += AT_NT) {
      const int g = i / (D / 2), f = i - g * (D / 2);
      const T* q = static_cast<const T*>(p.q) + ((size_t)b * p.Hq + h * G + g) * D + 2 * f;
      const float2 cs = rope_cos_sin(p.rope_turns[f], p.pos[b]);
      const float x0 = to_f32<T>(q[0]), x1 = to_f32<T>(q[1]);
      qs[g * D + 2 * f] = (x0 * cs.x - x1 * cs.y) * p.scale;
      qs[g * D + 2 * f + 1] = (x0 * cs.y + x1 * cs.x) * p.scale;
    }
    __syncthreads();
    float m[G_MAX], l[G_MAX], o[G_MAX][E];
#pragma unroll
    for (int g = 0; g < G_MAX; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[g][e] = 0.f;
    }
    for (int x = sg.x + warp; x < sg.seg_end(); x += AT_NW) {
      const int t0 = (x - sg.unit_begin) * PAGED_GROUP, n = min(PAGED_GROUP, len - t0);
      const int page = p.page_table[(size_t)b * p.max_pages + (t0 >> p.log2_page)];
      const long long row = paged_row(page, p.n_pages, p.Hkv, h, p.log2_page, t0);
      if (row < 0 && lane == 0) atomicOr(p.status, 1);
      for (int i = 0; i < n; ++i) {
        float k[E], v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          k[e] = row < 0 ? 0.f : to_f32<T>(static_cast<const T*>(p.k_pages)[(size_t)(row + i) * D + lane * E + e]);
          v[e] = row < 0 ? 0.f : to_f32<T>(static_cast<const T*>(p.v_pages)[(size_t)(row + i) * D + lane * E + e]);
        }
#pragma unroll
        for (int g = 0; g < G_MAX; ++g) {
          if (g >= G) break;
          float z = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) z += qs[g * D + lane * E + e] * k[e];
#pragma unroll
          for (int s = 16; s; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
          if (row < 0) z = -INFINITY;
          if (p.weight && lane == 0) p.logits[((size_t)unit * G + g) * p.T_cap + t0 + i] = z;
          const float mn = fmaxf(m[g], z);
          const float ms = mn == -INFINITY ? 0.f : mn;
          const float a = exp2f(m[g] - ms), w = exp2f(z - ms);
          m[g] = mn;
          l[g] = l[g] * a + w;
#pragma unroll
          for (int e = 0; e < E; ++e) o[g][e] = o[g][e] * a + w * v[e];
        }
      }
    }
    // the warps' parts, in warp order
#pragma unroll
    for (int g = 0; g < G_MAX; ++g) {
      if (g >= G) break;
#pragma unroll
      for (int e = 0; e < E; ++e) mrg[(warp * G + g) * D + lane * E + e] = o[g][e];
      if (lane == 0) {
        mml[(warp * G + g) * 2] = m[g];
        mml[(warp * G + g) * 2 + 1] = l[g];
      }
    }
    __syncthreads();
    const bool whole = sg.x == sg.unit_begin && sg.unit_end <= r1;
    float* rec = p.records + (size_t)(2 * c + (sg.unit_begin < r0 ? 0 : 1)) * paged_record_floats(G, D);
    for (int i = tid; i < G * D; i += AT_NT) {
      const int g = i / D;
      float M = -INFINITY;
      for (int w = 0; w < AT_NW; ++w) M = fmaxf(M, mml[(w * G + g) * 2]);
      const float Ms = M == -INFINITY ? 0.f : M;
      float L = 0.f, O = 0.f;
      for (int w = 0; w < AT_NW; ++w) {
        const float a = exp2f(mml[(w * G + g) * 2] - Ms);
        L += mml[(w * G + g) * 2 + 1] * a;
        O += mrg[w * G * D + i] * a;
      }
      if (whole) {
        p.out[((size_t)b * p.Hq + h * G) * D + i] = L > 0.f ? O / L : 0.f;
        if (p.weight && i == g * D) p.lse[(size_t)unit * G + g] = L > 0.f ? M + log2f(L) : INFINITY;
      } else {
        rec[i] = O;
        if (i == g * D) {
          rec[G * D + g] = M;
          rec[G * D + G + g] = L;
        }
      }
    }
    if (tid == 0 && sg.unit_begin >= r0 && sg.unit_end > r1)
      p.joins[c] = make_int2(unit, paged_part_of(total, parts, sg.unit_end - 1));
    __syncthreads();
    sg.next();
  }
}

// log2 of a cut unit's softmax denominator, from its parts' records: thread g.
__device__ float joined_lse(const PagedAttendParams& p, int D, int g, int c0, int c1) {
  const int R = paged_record_floats(p.G, D);
  float M = -INFINITY, L = 0.f;
  for (int c = c0; c <= c1; ++c) M = fmaxf(M, p.records[(size_t)(2 * c + (c == c0)) * R + p.G * D + g]);
  const float Ms = M == -INFINITY ? 0.f : M;
  for (int c = c0; c <= c1; ++c) {
    const float* r = p.records + (size_t)(2 * c + (c == c0)) * R + p.G * D;
    L += r[p.G + g] * exp2f(r[g] - Ms);
  }
  return L > 0.f ? M + log2f(L) : INFINITY;
}

// Block c: the unit that begins in part c and goes on; with weights then its
// share of the line's tokens.
template <int D>
__global__ void __launch_bounds__(AT_NT) paged_join_kernel(const __grid_constant__ PagedAttendParams p) {
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, c = blockIdx.x, G = p.G;
  const int2 jn = c < p.grid ? p.joins[c] : make_int2(-1, 0);
  if (jn.x >= 0) {
    const int R = paged_record_floats(G, D);
    for (int i = tid; i < G * D; i += AT_NT) {
      const int g = i / D;
      float M = -INFINITY, L = 0.f, O = 0.f;
      for (int k = c; k <= jn.y; ++k) M = fmaxf(M, p.records[(size_t)(2 * k + (k == c)) * R + G * D + g]);
      const float Ms = M == -INFINITY ? 0.f : M;
      for (int k = c; k <= jn.y; ++k) {
        const float* r = p.records + (size_t)(2 * k + (k == c)) * R;
        const float a = exp2f(r[G * D + g] - Ms);
        L += r[G * D + G + g] * a;
        O += r[i] * a;
      }
      const int b = jn.x / p.Hkv, h = jn.x - b * p.Hkv;
      p.out[((size_t)b * p.Hq + h * G) * D + i] = L > 0.f ? O / L : 0.f;
    }
  }
  if (!p.weight) return;
  float* lse = sm;
  int* scan = reinterpret_cast<int*>(sm + G_MAX);
  int* pre = scan + 32;
  group_prefix<AT_NT>(p, pre, scan, false);
  const int total = pre[p.B] * p.Hkv;
  const int parts = paged_parts(total, p.grid);
  const int blocks = min((int)gridDim.x, max(total, 1));
  if (c >= blocks || total == 0) return;
  Segments sg;
  sg.start(pre, p.B, p.Hkv, paged_part_begin(total, blocks, c), paged_part_begin(total, blocks, c + 1));
  while (sg.at()) {
    const int unit = sg.b * p.Hkv + sg.h, len = clamped_len(p, sg.b);
    const int c0 = paged_part_of(total, parts, sg.unit_begin), c1 = paged_part_of(total, parts, sg.unit_end - 1);
    __syncthreads();
    if (tid < G) lse[tid] = c0 == c1 ? p.lse[(size_t)unit * G + tid] : joined_lse(p, D, tid, c0, c1);
    __syncthreads();
    const int t1 = min(len, (sg.seg_end() - sg.unit_begin) * PAGED_GROUP);
    for (int t = (sg.x - sg.unit_begin) * PAGED_GROUP + tid; t < t1; t += AT_NT) {
      float w = 0.f;
      for (int g = 0; g < G; ++g) w += exp2f(p.logits[((size_t)unit * G + g) * p.T_cap + t] - lse[g]);
      p.weight[(size_t)unit * p.T_cap + t] += w;
    }
    sg.next();
  }
}

template <typename T, int D>
cudaError_t launch(const PagedAttendParams& p, cudaStream_t s) {
  const int smem = (G_MAX * D + AT_NW * G_MAX * (D + 2)) * 4 + 32 * 4 + (p.B + 1) * 4;
  cudaError_t e = cudaFuncSetAttribute(paged_attend_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  paged_attend_kernel<T, D><<<p.grid, AT_NT, smem, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  paged_join_kernel<D><<<p.weight ? 4 * p.grid : p.grid, AT_NT, G_MAX * 4 + 32 * 4 + (p.B + 1) * 4, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_attend(const PagedAttendParams& p0, int head_dim, bool bf16, int sms, cudaStream_t s) {
  PagedAttendParams p = p0;
  p.grid = min(sms, PAGED_MAX_PARTS);
  using B16 = __nv_bfloat16;
  if (bf16) return head_dim == 128 ? launch<B16, 128>(p, s) : launch<B16, 64>(p, s);
  return head_dim == 128 ? launch<float, 128>(p, s) : launch<float, 64>(p, s);
}

}  // namespace fasa
