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
#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <mutex>

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

// ------------------------------------------------------ bf16: tensor cores
// A warp takes a group of 16 tokens at a time, through a ring of its own in
// shared memory that TMA fills (one copy of 16 rows for K, one for V, in the
// 128-byte swizzle, so that ldmatrix reads without bank conflicts), and no
// warp waits for another before a unit's end.
//   z^T: rows of A the heads, B the tokens.  The rotated and scaled query is
//   three bf16 terms (24 bits: the logits are as exact as fp32's), the first
//   two as rows 0-7 and 8-15 of one operand, the third as another.
//   o^T = V^T P^T: the z fragment is the P fragment of the same lane, in two
//   bf16 terms (16 bits of a weight that is summed with others), V read
//   transposed.
constexpr int TC_NW = 8;
constexpr int TC_NT = TC_NW * 32;

template <int D>
struct Tc {
  static constexpr int HALF = PAGED_GROUP * 128;        // bytes of 64 columns of a group
  static constexpr int ROWS = (D / 64) * HALF;          // K or V of a group
  static constexpr int STAGE = 2 * ROWS;
  static constexpr int STAGES = 196608 / (TC_NW * STAGE);
  static constexpr int MT = D / 16;
  static constexpr int OREGS = 4 * MT;
  // shared memory, from a 1024-byte boundary
  static constexpr int OFF_MRG = TC_NW * STAGES * STAGE;             // [4][OREGS][32] floats
  static constexpr int OFF_ML = OFF_MRG + 4 * OREGS * 32 * 4;        // [4][8] (m, l)
  static constexpr int OFF_CS = OFF_ML + 4 * 8 * 8;                  // [D/2] (cos, sin)
  static constexpr int OFF_TURNS = OFF_CS + D / 2 * 8;
  static constexpr int OFF_BAR = OFF_TURNS + D / 2 * 8;
  static constexpr int OFF_HELD = OFF_BAR + TC_NW * STAGES * 8;      // whether a stage's page is in the pool
  static constexpr int OFF_SCAN = OFF_HELD + TC_NW * STAGES * 4;
  static constexpr int OFF_PRE = OFF_SCAN + 32 * 4;
};

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(map), "r"(0), "r"(row), "r"(0), "r"(bar)
      : "memory");
}

template <int D>
__global__ void __launch_bounds__(TC_NT, 1)
    paged_attend_bf16_kernel(const __grid_constant__ PagedAttendParams p, const __grid_constant__ CUtensorMap kmap,
                             const __grid_constant__ CUtensorMap vmap) {
  using C = Tc<D>;
  constexpr int S = C::STAGES, MT = C::MT;
  extern __shared__ __align__(16) char raw[];
  char* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int G = p.G;
  float* mrg = reinterpret_cast<float*>(sm + C::OFF_MRG);
  float2* ml = reinterpret_cast<float2*>(sm + C::OFF_ML);
  float2* cs = reinterpret_cast<float2*>(sm + C::OFF_CS);
  unsigned long long* turns = reinterpret_cast<unsigned long long*>(sm + C::OFF_TURNS);
  int* held = reinterpret_cast<int*>(sm + C::OFF_HELD) + warp * S;
  int* scan = reinterpret_cast<int*>(sm + C::OFF_SCAN);
  int* pre = reinterpret_cast<int*>(sm + C::OFF_PRE);
  const uint32_t ring = smem_u32(sm) + warp * S * C::STAGE;
  const uint32_t bars = smem_u32(sm + C::OFF_BAR) + warp * S * 8;
  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(bars + 8 * i, 1);
    fence_mbar_init();
  }
  // (lanes reading different parameter words take turns: a few lanes of each warp)
  if (lane < D / 2 / TC_NW) turns[warp * (D / 2 / TC_NW) + lane] = p.rope_turns[warp * (D / 2 / TC_NW) + lane];
  group_prefix<TC_NT>(p, pre, scan, blockIdx.x == 0);
  const int total = pre[p.B] * p.Hkv;
  const int parts = paged_parts(total, p.grid);
  const int c = blockIdx.x;
  for (int b = c; b < p.B; b += p.grid)  // sequences without a token: zeros
    if (pre[b] == pre[b + 1])
      for (int i = tid; i < p.Hq * D; i += TC_NT) p.out[(size_t)b * p.Hq * D + i] = 0.f;
  if (tid == 0) p.joins[c] = make_int2(-1, 0);
  if (c >= parts) return;
  const int r0 = paged_part_begin(total, parts, c), r1 = paged_part_begin(total, parts, c + 1);

  // This warp's groups: x = r0 + warp + k * TC_NW, k < mine.  Lane i holds the
  // pool row of group (batch of 32) + i.
  const int mine = max(0, (r1 - r0 - warp + TC_NW - 1) / TC_NW);
  int rows = -1, issued = 0;
  bool dead = false;  // a wait ran out: nothing more is copied or waited for
  auto look_up = [&](int k) {
    const int x = r0 + warp + (k + lane) * TC_NW;
    rows = -1;
    if (k + lane < mine) {
      const int b = sequence_of(pre, p.B, p.Hkv, x);
      const int n = pre[b + 1] - pre[b], rem = x - pre[b] * p.Hkv;
      const int h = rem / n, slot = (rem - h * n) * PAGED_GROUP;
      const int page = __ldg(p.page_table + (size_t)b * p.max_pages + (slot >> p.log2_page));
      rows = (int)paged_row(page, p.n_pages, p.Hkv, h, p.log2_page, slot);
      if (rows < 0) atomicOr(p.status, 1);
    }
  };
  auto issue = [&]() {  // the next group of this warp, into its stage
    if (issued >= mine || dead) return;
    if ((issued & 31) == 0) look_up(issued);
    const int row = __shfl_sync(0xffffffffu, rows, issued & 31);
    const int st = issued % S;
    if (lane == 0) {
      held[st] = row >= 0;
      const uint32_t bar = bars + 8 * st, dst = ring + st * C::STAGE;
      if (row >= 0) {
        mbar_arrive_expect_tx(bar, C::STAGE);
        tma_rows(dst, &kmap, row, bar);
        tma_rows(dst + C::ROWS, &vmap, row, bar);
      } else {
        mbar_arrive(bar);
      }
    }
    ++issued;
  };
  for (int i = 0; i < S; ++i) issue();

  // ldmatrix: lane's row of the group and 16-byte chunk of a 16-column slab
  const int lrow = (lane & 7) + ((lane >> 4) << 3), lch = (lane >> 3) & 1;
  auto chunk_at = [&](int slab) {  // byte offset in K or V of a group
    const int ch = 2 * slab + lch;
    return (ch >> 3) * C::HALF + lrow * 128 + (((ch & 7) ^ (lrow & 7)) << 4);
  };

  Segments sg;
  sg.start(pre, p.B, p.Hkv, r0, r1);
  int k = 0, cur_b = -1;
  while (sg.at()) {
    const int b = sg.b, h = sg.h, unit = b * p.Hkv + h;
    const int len = clamped_len(p, b);
    if (b != cur_b) {
      for (int f = tid; f < D / 2; f += TC_NT) {
        const float2 a = rope_cos_sin(turns[f], p.pos[b]);
        cs[f] = make_float2(a.x * p.scale, a.y * p.scale);
      }
      cur_b = b;
      __syncthreads();
    }
    // the query fragments: three terms of q of head g, zeros behind the last head
    uint32_t qa[MT][4], ql[MT][2];
    {
      const uint32_t* q = static_cast<const uint32_t*>(p.q) + ((size_t)b * p.Hq + h * G + min(g, G - 1)) * (D / 2);
#pragma unroll
      for (int s = 0; s < MT; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int f = 8 * s + t + 4 * e;
          const uint32_t w = g < G ? __ldg(q + f) : 0u;
          const float2 a = cs[f];
          const float x0 = bf16_lo(w), x1 = bf16_hi(w);
          const float y0 = x0 * a.x - x1 * a.y, y1 = x0 * a.y + x1 * a.x;
          const uint32_t hi = pack_bf16(y0, y1);
          const float u0 = y0 - bf16_lo(hi), u1 = y1 - bf16_hi(hi);
          split_bf16(u0, u1, qa[s][2 * e + 1], ql[s][e]);
          qa[s][2 * e] = hi;
        }
    }
    float m = -INFINITY, l = 0.f, o[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float* logits = p.weight ? p.logits + ((size_t)unit * G + g) * p.T_cap + 2 * t : nullptr;

    for (; k < mine && r0 + warp + k * TC_NW < sg.seg_end(); ++k) {
      const int t0 = (r0 + warp + k * TC_NW - sg.unit_begin) * PAGED_GROUP;
      const int st = k % S;
      const uint32_t kb = ring + st * C::STAGE, vb = kb + C::ROWS;
      if (!dead && !mbar_wait_bounded(bars + 8 * st, (k / S) & 1, p.wait_ns)) {
        if (lane == 0) atomicOr(p.status, 2);
        dead = true;
      }
      dead = __any_sync(0xffffffffu, dead);
      __syncwarp();
      const int n = held[st] && !dead ? min(PAGED_GROUP, len - t0) : 0;
      if (n < PAGED_GROUP) {  // what lies behind the end counts for nothing, NaN neither
        for (int i = lane; i < (PAGED_GROUP - n) * (D / 8); i += 32) {
          const int r = n + i / (D / 8), ch = i % (D / 8);
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vb + (ch >> 3) * C::HALF + r * 128 + ((ch & 7) << 4)),
                       "r"(0)
                       : "memory");
        }
        fence_proxy_async();
        __syncwarp();
      }
      float za[2][4] = {}, zb[2][4] = {};
#pragma unroll
      for (int s = 0; s < MT; ++s) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4(kb + chunk_at(s), b0, b1, b2, b3);
        mma_bf16_16816(za[0], qa[s][0], qa[s][1], qa[s][2], qa[s][3], b0, b1);
        mma_bf16_16816(za[1], qa[s][0], qa[s][1], qa[s][2], qa[s][3], b2, b3);
        mma_bf16_16816(zb[0], ql[s][0], 0u, ql[s][1], 0u, b0, b1);
        mma_bf16_16816(zb[1], ql[s][0], 0u, ql[s][1], 0u, b2, b3);
      }
      float z[4];  // head g, tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[i] = (zb[i >> 1][i & 1] + za[i >> 1][2 + (i & 1)]) + za[i >> 1][i & 1];
        if (2 * t + (i & 1) + 8 * (i >> 1) >= n) z[i] = -INFINITY;
      }
      if (logits && g < G) {
        *reinterpret_cast<float2*>(logits + t0) = make_float2(z[0], z[1]);
        *reinterpret_cast<float2*>(logits + t0 + 8) = make_float2(z[2], z[3]);
      }
      float mx = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (__any_sync(0xffffffffu, mx > m)) {
        const float mn = fmaxf(m, mx);
        const float a = mn == -INFINITY ? 1.f : exp2f(m - mn);
        m = mn;
        l *= a;
        const float a0 = __shfl_sync(0xffffffffu, a, 8 * t), a1 = __shfl_sync(0xffffffffu, a, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          o[i][0] *= a0;
          o[i][1] *= a1;
          o[i][2] *= a0;
          o[i][3] *= a1;
        }
      }
      const float ms = m == -INFINITY ? 0.f : m;
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = exp2f(z[i] - ms);
        l += w[i];
      }
      uint32_t h0, h1, l0, l1;
      split_bf16(w[0], w[1], h0, l0);
      split_bf16(w[2], w[3], h1, l1);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        uint32_t a0, a1, a2, a3;
        ldsm_x4_t(vb + chunk_at(i), a0, a1, a2, a3);
        mma_bf16_16816(o[i], a0, a1, a2, a3, h0, h1);
        mma_bf16_16816(o[i], a0, a1, a2, a3, l0, l1);
      }
      __syncwarp();
      issue();
    }

    // the eight warps' parts: 4-7 into 0-3 lane by lane, then four records
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    float* dump = mrg + (warp & 3) * C::OREGS * 32 + lane;
    auto put = [&]() {
#pragma unroll
      for (int i = 0; i < C::OREGS; ++i) dump[i * 32] = o[i >> 2][i & 3];
      if (t == 0) ml[(warp & 3) * 8 + g] = make_float2(m, l);
    };
    if (warp >= 4) put();
    __syncthreads();
    if (warp < 4) {
      const float2 other = ml[warp * 8 + g];
      const float M = fmaxf(m, other.x), Ms = M == -INFINITY ? 0.f : M;
      const float a = exp2f(m - Ms), e = exp2f(other.x - Ms);
      m = M;
      l = l * a + other.y * e;
      const float a0 = __shfl_sync(0xffffffffu, a, 8 * t), a1 = __shfl_sync(0xffffffffu, a, 8 * t + 4);
      const float e0 = __shfl_sync(0xffffffffu, e, 8 * t), e1 = __shfl_sync(0xffffffffu, e, 8 * t + 4);
#pragma unroll
      for (int i = 0; i < C::OREGS; ++i)
        o[i >> 2][i & 3] = o[i >> 2][i & 3] * ((i & 1) ? a1 : a0) + dump[i * 32] * ((i & 1) ? e1 : e0);
      __syncwarp();
      put();
    }
    __syncthreads();
    const bool whole = sg.x == sg.unit_begin && sg.unit_end <= r1;
    float* rec = p.records + (size_t)(2 * c + (sg.unit_begin < r0 ? 0 : 1)) * paged_record_floats(G, D);
    for (int i = tid; i < C::OREGS * 32; i += TC_NT) {
      const int ln = i & 31, e = (i >> 5) & 3;
      const int hd = (ln & 3) * 2 + (e & 1), dim = (i >> 7) * 16 + (ln >> 2) + (e >> 1) * 8;
      if (hd >= G) continue;
      float2 r[4];
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        r[w] = ml[w * 8 + hd];
        M = fmaxf(M, r[w].x);
      }
      const float Ms = M == -INFINITY ? 0.f : M;
      float L = 0.f, O = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float a = exp2f(r[w].x - Ms);
        L += r[w].y * a;
        O += mrg[w * C::OREGS * 32 + i] * a;
      }
      if (whole) {
        p.out[((size_t)b * p.Hq + h * G + hd) * D + dim] = L > 0.f ? O / L : 0.f;
        if (p.weight && dim == 0) p.lse[(size_t)unit * G + hd] = L > 0.f ? M + log2f(L) : INFINITY;
      } else {
        rec[hd * D + dim] = O;
        if (dim == 0) {
          rec[G * D + hd] = M;
          rec[G * D + G + hd] = L;
        }
      }
    }
    if (tid == 0 && sg.unit_begin >= r0 && sg.unit_end > r1)
      p.joins[c] = make_int2(unit, paged_part_of(total, parts, sg.unit_end - 1));
    __syncthreads();
    sg.next();
  }
  // after a wait that ran out: no copy may land in memory of a block that is gone
  if (dead)
    for (; k < issued; ++k)
      if (!mbar_wait_bounded(bars + 8 * (k % S), (k / S) & 1, p.wait_ns) && lane == 0) atomicOr(p.status, 4);
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

// A pool of pages as rows of 64-column halves: a copy takes a group's 16 rows.
cudaError_t pool_map(CUtensorMap* map, const void* pool, long long rows, int D) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::mutex mu;
  static Encode encode = nullptr;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!encode) {
      void* f = nullptr;
      cudaDriverEntryPointQueryResult found;
      const cudaError_t e =
          cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
      if (e != cudaSuccess) return e;
      if (found != cudaDriverEntryPointSuccess || !f) return cudaErrorSymbolNotFound;
      encode = reinterpret_cast<Encode>(f);
    }
  }
  const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(D / 64)};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, 128};
  const cuuint32_t box[3] = {64, PAGED_GROUP, (cuuint32_t)(D / 64)}, one[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(pool), dims, strides, box, one,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D>
cudaError_t join(const PagedAttendParams& p, cudaStream_t s) {
  paged_join_kernel<D><<<p.weight ? 4 * p.grid : p.grid, AT_NT, G_MAX * 4 + 32 * 4 + (p.B + 1) * 4, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_f32(const PagedAttendParams& p, cudaStream_t s) {
  const int smem = (G_MAX * D + AT_NW * G_MAX * (D + 2)) * 4 + 32 * 4 + (p.B + 1) * 4;
  cudaError_t e = cudaFuncSetAttribute(paged_attend_kernel<float, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  paged_attend_kernel<float, D><<<p.grid, AT_NT, smem, s>>>(p);
  e = cudaGetLastError();
  return e == cudaSuccess ? join<D>(p, s) : e;
}

template <int D>
cudaError_t launch_bf16(const PagedAttendParams& p, cudaStream_t s) {
  CUtensorMap km, vm;
  const long long rows = ((long long)p.n_pages * p.Hkv) << p.log2_page;
  cudaError_t e = pool_map(&km, p.k_pages, rows, D);
  if (e == cudaSuccess) e = pool_map(&vm, p.v_pages, rows, D);
  if (e != cudaSuccess) return e;
  const int smem = 1024 + Tc<D>::OFF_PRE + (p.B + 1) * 4;
  e = cudaFuncSetAttribute(paged_attend_bf16_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  paged_attend_bf16_kernel<D><<<p.grid, TC_NT, smem, s>>>(p, km, vm);
  e = cudaGetLastError();
  return e == cudaSuccess ? join<D>(p, s) : e;
}

}  // namespace

cudaError_t launch_paged_attend(const PagedAttendParams& p0, int head_dim, bool bf16, int sms, cudaStream_t s) {
  PagedAttendParams p = p0;
  p.grid = min(sms, PAGED_MAX_PARTS);
  if (bf16) return head_dim == 128 ? launch_bf16<128>(p, s) : launch_bf16<64>(p, s);
  return head_dim == 128 ? launch_f32<128>(p, s) : launch_f32<64>(p, s);
}

}  // namespace fasa
