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
// attend: each warp takes one part of the line of all token groups
// (fasa_paged_index.h), unit by unit, group by group, with a running (m, l, o).
// A unit it holds whole is finished there; otherwise its record goes to the
// workspace.  join: the records of a unit that was cut, in a fixed order; and
// with weights, a second pass over the logits the first one left.
//
// The bytes of K and V bound it, so a warp's groups come through a ring of its
// own in shared memory that TMA fills (one copy of 16 rows for K, one for V, in
// the 128-byte swizzle: no bank conflicts), page by page wherever the pages
// lie, and no warp waits for another: what a unit costs beside its bytes is
// hidden by the other warps of the SM.
#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "fasa_cluster.cuh"
#include "fasa_internal.h"
#include "fasa_paged.h"
#include "fasa_ptx.cuh"

namespace fasa {
namespace {

constexpr int JN_NT = 256;  // threads of a join block

// The line's words, in shared memory.  Every thread of the block calls it; ends
// with a barrier.  scan: NT / 32 words.  A batch of more than NT sequences has its
// lengths read at once and a run of them to a thread (1024 of 48 tokens: 53.9 us, 55.2
// with NT at a time).
template <int NT>
__device__ void make_line(const PagedCommon& p, unsigned* w, int* scan, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // (past L1: the join reads them ahead of its wait, when its SM's L1 may hold what
  // they were before the kernel in front of the attention wrote them)
  bool bad = false;
  auto length = [&](int b) {
    const int len = ld_cg(p.seq_lens + b);
    bad = bad || len < 0 || len > p.T_cap;
    return min(max(len, 0), p.T_cap);
  };
  const bool many = p.B > NT;
  const int run = ((p.B + NT - 1) / NT) | 1;  // (odd: its threads' words lie in as many banks)
  const int b0 = tid * run, b1 = min(p.B, b0 + run);
  int len = 0, groups = 0;
  if (!many) {
    if (tid < p.B) len = length(tid);
    groups = paged_groups(len);
  } else {
#pragma unroll 8
    for (int b = tid; b < p.B; b += NT) w[b] = (unsigned)length(b);
    __syncthreads();
    for (int b = b0; b < b1; ++b) groups += paged_groups((int)w[b]);
  }
  if (report && bad) atomicOr(p.status, 1);
  int incl = groups;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int before = incl - groups;
#pragma unroll
  for (int v = 0; v < NT / 32; ++v) before += v < warp ? scan[v] : 0;
  if (tid == NT - 1) w[p.B] = paged_word(before + groups, 0);
  if (!many) {
    if (tid < p.B) w[tid] = paged_word(before, len);
  } else {
    for (int b = b0; b < b1; ++b) {
      len = (int)w[b];
      w[b] = paged_word(before, len);
      before += paged_groups(len);
    }
  }
  __syncthreads();
}

// x0, x1 as bf16 pairs hi + mid + lo: 24 bits and more of each.
__device__ __forceinline__ void split3_bf16(float x0, float x1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack_bf16(x0, x1);
  split_bf16(x0 - bf16_lo(hi), x1 - bf16_hi(hi), mid, lo);
}

// The logits of a group, where there are weights to add to: to[head][16], kept in
// L2 by `policy` until the join has read them.
struct Logits {
  float* to;
  unsigned long long policy;
  __device__ void put(int i, float a) const {
    asm volatile("st.global.L2::cache_hint.f32 [%0], %1, %2;" ::"l"(to + i), "f"(a), "l"(policy) : "memory");
  }
  __device__ void put(int i, float a, float b) const {
    asm volatile("st.global.L2::cache_hint.v2.f32 [%0], {%1, %2}, %3;" ::"l"(to + i), "f"(a), "f"(b), "l"(policy)
                 : "memory");
  }
};

// ------------------------------------------------- bf16: tensor cores
// z^T: rows of A the heads, B the tokens.  The rotated and scaled query is
// three bf16 terms (24 bits: the logits are as exact as fp32's).  o^T = V^T P^T:
// the z fragment is the P fragment of the same lane, in three bf16 terms too (two,
// 16 bits, left an error of 1e-6 where few tokens carry the sum), V read
// transposed.  Lane (g, t) = (lane / 4, lane % 4) holds the m of row g's head and
// its share of l, and of o the heads of the columns 2t, 2t + 1 at the dims 16 i + g,
// 16 i + g + 8.
// PACK, for at most four heads: the rows 0-3, 4-7, 8-11 of one operand are a head's
// terms, and of P's columns 0-3 the first terms, 4-7 the second: 32 instructions a
// group instead of 56, which a part's last group waits for.
template <int D, bool PACK>
struct MathBf16 {
  using T = __nv_bfloat16;
  static constexpr int CTAS = 2;  // per SM
  // Warps of a CTA.  Two with six stages each read 128 dims at the copy
  // rate (344.4 us for 2.38 GB) and leave half the records to join that four with
  // three do (350.6 us); a group of 64 dims is half the bytes for the same
  // latency and wants the four (64 short sequences: 17.7 us against 23.6).
  static constexpr int WARPS = D == 128 ? 2 : 4;
  static constexpr int RAW = G_MAX * D * 2;  // the next unit's raw query, fetched while this one is read
  static constexpr int MT = D / 16;
  static constexpr int SCRATCH = 0;  // shared memory of a warp
  static constexpr CUtensorMapDataType TYPE = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  uint32_t qa[MT][4], ql[PACK ? 1 : MT][2];
  float m, l, o[MT][4];

  // query: the unit's raw rows [G][D].
  __device__ void begin(const void* query, const float2* cs, int G, float*) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3, head = PACK ? g & 3 : g;
    const uint32_t* raw = static_cast<const uint32_t*>(query) + min(head, G - 1) * (D / 2);
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {  // the pairs t + 4 i of the head
      const float2 a = cs[t + 4 * i];
      const uint32_t w = head < G ? raw[t + 4 * i] : 0u;
      const float x0 = bf16_lo(w), x1 = bf16_hi(w);
      const float y0 = x0 * a.x - x1 * a.y, y1 = x0 * a.y + x1 * a.x;
      uint32_t hi, mid, lo;
      split3_bf16(y0, y1, hi, mid, lo);
      if constexpr (PACK) {
        qa[i >> 1][2 * (i & 1)] = g < 4 ? hi : mid;
        qa[i >> 1][2 * (i & 1) + 1] = g < 4 ? lo : 0u;
      } else {
        qa[i >> 1][2 * (i & 1)] = hi;
        qa[i >> 1][2 * (i & 1) + 1] = mid;
        ql[i >> 1][i & 1] = lo;
      }
    }
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < 4 * MT; ++i) o[i >> 2][i & 3] = 0.f;
  }
  __device__ void scale_o(float a) {
    const int t = threadIdx.x & 3;
    const float a0 = __shfl_sync(0xffffffffu, a, 8 * t), a1 = __shfl_sync(0xffffffffu, a, 8 * t + 4);
#pragma unroll
    for (int i = 0; i < 4 * MT; ++i) o[i >> 2][i & 3] *= (i & 1) ? a1 : a0;
  }
  // One group: K at kb, V at vb, its first n tokens count.
  __device__ void step(uint32_t kb, uint32_t vb, int n, const Logits& logits, int G, float*) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // ldmatrix: this lane's row of the group and 16-byte chunk of a 16-column slab
    const int lrow = (lane & 7) + ((lane >> 4) << 3), lch = (lane >> 3) & 1;
    auto chunk_at = [&](int slab) {
      const int ch = 2 * slab + lch;
      return (ch >> 3) * (PAGED_GROUP * 128) + lrow * 128 + (((ch & 7) ^ (lrow & 7)) << 4);
    };
    // (sums of their own for the even slabs, the odd ones and the third term: shorter
    // chains, and less of the accumulator's rounding towards zero)
    float za[2][2][4] = {}, zb[PACK ? 1 : 2][4] = {};
#pragma unroll
    for (int s = 0; s < MT; ++s) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4(kb + chunk_at(s), b0, b1, b2, b3);
      mma_bf16_16816(za[s & 1][0], qa[s][0], qa[s][1], qa[s][2], qa[s][3], b0, b1);
      mma_bf16_16816(za[s & 1][1], qa[s][0], qa[s][1], qa[s][2], qa[s][3], b2, b3);
      if constexpr (!PACK) {
        mma_bf16_16816(zb[0], ql[s][0], 0u, ql[s][1], 0u, b0, b1);
        mma_bf16_16816(zb[1], ql[s][0], 0u, ql[s][1], 0u, b2, b3);
      }
    }
    float z[4];  // the head's, tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int nt = i >> 1, e = i & 1;
      const float low = za[0][nt][2 + e] + za[1][nt][2 + e], high = za[0][nt][e] + za[1][nt][e];
      if constexpr (PACK) {
        z[i] = low + high;
        z[i] += __shfl_xor_sync(0xffffffffu, z[i], 16);
      } else {
        z[i] = (zb[nt][e] + low) + high;
      }
      if (2 * t + (i & 1) + 8 * (i >> 1) >= n) z[i] = -INFINITY;
    }
    if (logits.to && g < G) {
      logits.put(g * PAGED_GROUP + 2 * t, z[0], z[1]);
      logits.put(g * PAGED_GROUP + 2 * t + 8, z[2], z[3]);
    }
    float mx = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    if (__any_sync(0xffffffffu, mx > m)) {
      const float mn = fmaxf(m, mx);
      const float a = mn == -INFINITY ? 1.f : exp2f(m - mn);
      m = mn;
      l *= a;
      scale_o(a);
    }
    const float ms = m == -INFINITY ? 0.f : m;
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = exp2f(z[i] - ms);
      l += w[i];
    }
    uint32_t h0, h1, m0, m1, l0, l1;
    split3_bf16(w[0], w[1], h0, m0, l0);
    split3_bf16(w[2], w[3], h1, m1, l1);
    if constexpr (PACK) {  // column g: the first term, or head g - 4's second
      h0 = g < 4 ? h0 : m0;
      h1 = g < 4 ? h1 : m1;
      l0 = g < 4 ? l0 : 0u;
      l1 = g < 4 ? l1 : 0u;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      uint32_t a0, a1, a2, a3;
      ldsm_x4_t(vb + chunk_at(i), a0, a1, a2, a3);
      // (a sum of its own: the tensor cores' accumulator rounds towards zero, which
      // over the thousands of groups of a long part would add up)
      float acc[4] = {};
      mma_bf16_16816(acc, a0, a1, a2, a3, l0, l1);
      if constexpr (!PACK) mma_bf16_16816(acc, a0, a1, a2, a3, m0, m1);
      mma_bf16_16816(acc, a0, a1, a2, a3, h0, h1);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] += acc[e];
    }
  }
  // l of a head in all its lanes, o whole.
  __device__ void finish() {
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if constexpr (PACK) {
#pragma unroll
      for (int i = 0; i < 4 * MT; ++i) o[i >> 2][i & 3] += __shfl_xor_sync(0xffffffffu, o[i >> 2][i & 3], 2);
    }
  }
  // (m, l) of head g to ml(g, m, l), by one lane; o times inv (by head) to to[head][dim].
  template <class F>
  __device__ void stats(int G, F&& ml) const {
    const int lane = threadIdx.x & 31;
    if ((lane & 3) == 0 && (lane >> 2) < G) ml(lane >> 2, m, l);
  }
  __device__ void write(float* to, int G, bool divide) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const float inv = !divide ? 1.f : l > 0.f ? 1.f / l : 0.f;
    const float i0 = __shfl_sync(0xffffffffu, inv, 8 * t), i1 = __shfl_sync(0xffffffffu, inv, 8 * t + 4);
#pragma unroll
    for (int i = 0; i < 4 * MT; ++i) {
      const int head = 2 * t + (i & 1);
      if (head < G) to[head * D + (i >> 2) * 16 + g + ((i >> 1) & 1) * 8] = o[i >> 2][i & 3] * ((i & 1) ? i1 : i0);
    }
  }
};

// ------------------------------------------------- fp32: CUDA cores
// Lane (token, half) = (lane % 16, lane / 16) takes half of the dims of its
// token's logits, K four dims at a time from its row and the query's from an
// address all tokens share; for o a lane holds D / 32 dims of every head and
// reads the weights of a token as a broadcast.  GP: heads in registers, 4 or 8.
template <int D, int GP>
struct MathF32 {
  using T = float;
  static constexpr int CTAS = 1;
  // Warps of a CTA: as many as hide the arithmetic's latency, then stages.  At 537 MB:
  // 4 heads of 64 dims 83.6 us with eight warps, 117.1 with four; 8 heads of 128 dims
  // 106.2 and 116.8 (one stage against three); 4 heads of 128 dims 86.7 and 82.8.
  static constexpr int WARPS = D == 128 && GP == 4 ? 4 : 8;
  static constexpr int RAW = 0;  // (no room to fetch ahead: the raw query goes where the turned one stays)
  static constexpr int E = D / 32;
  static constexpr int SCRATCH = (GP * D + PAGED_GROUP * GP) * 4;  // the query, a group's weights
  static constexpr CUtensorMapDataType TYPE = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  float m[GP], l[GP], o[GP][E];

  // The raw rows [G][D] are turned where they lie; zeros behind the last head.
  __device__ void begin(const void*, const float2* cs, int G, float* scratch) {
    float2* qs = reinterpret_cast<float2*>(scratch);
#pragma unroll 4
    for (int i = threadIdx.x & 31; i < GP * (D / 2); i += 32) {
      const float2 x = i < G * (D / 2) ? qs[i] : make_float2(0.f, 0.f), a = cs[i % (D / 2)];
      qs[i] = make_float2(x.x * a.x - x.y * a.y, x.x * a.y + x.y * a.x);
    }
    __syncwarp();
#pragma unroll
    for (int g = 0; g < GP; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[g][e] = 0.f;
    }
  }
  __device__ void step(uint32_t kb, uint32_t vb, int n, const Logits& logits, int G, float* scratch) {
    const int lane = threadIdx.x & 31, tok = lane & 15, half = lane >> 4;
    const float4* qs = reinterpret_cast<const float4*>(scratch) + half * (D / 8);
    float* ps = scratch + GP * D;
    float z[GP];
#pragma unroll
    for (int g = 0; g < GP; ++g) z[g] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
      const int ch = half * (D / 8) + c;
      float4 k;
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(k.x), "=f"(k.y), "=f"(k.z), "=f"(k.w)
                   : "r"(kb + (ch >> 3) * (PAGED_GROUP * 128) + tok * 128 + (((ch & 7) ^ (tok & 7)) << 4))
                   : "memory");
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        const float4 q = qs[g * (D / 4) + c];
        z[g] = fmaf(k.x, q.x, fmaf(k.y, q.y, fmaf(k.z, q.z, fmaf(k.w, q.w, z[g]))));
      }
    }
    bool up = false;
#pragma unroll
    for (int g = 0; g < GP; ++g) {
      z[g] += __shfl_xor_sync(0xffffffffu, z[g], 16);
      if (tok >= n) z[g] = -INFINITY;
      if (logits.to && g < G && half == 0) logits.put(g * PAGED_GROUP + tok, z[g]);
      up = up || z[g] > m[g];
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        float mn = fmaxf(m[g], z[g]);
#pragma unroll
        for (int s = 1; s < 16; s <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, s));
        const float a = mn == -INFINITY ? 1.f : exp2f(m[g] - mn);
        m[g] = mn;
        l[g] *= a;
#pragma unroll
        for (int e = 0; e < E; ++e) o[g][e] *= a;
      }
    }
    __syncwarp();  // the last group's weights are read
#pragma unroll
    for (int g = 0; g < GP; ++g) {
      const float w = exp2f(z[g] - (m[g] == -INFINITY ? 0.f : m[g]));
      if (half == 0) {
        l[g] += w;
        ps[tok * GP + g] = w;
      }
    }
    __syncwarp();
#pragma unroll 4
    for (int i = 0; i < PAGED_GROUP; ++i) {
      float v[E];
      const int ch = lane * E / 4;
      const uint32_t at = vb + (ch >> 3) * (PAGED_GROUP * 128) + i * 128 + (((ch & 7) ^ (i & 7)) << 4);
      if constexpr (E == 4)
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                     : "r"(at)
                     : "memory");
      else
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "r"(at + 8 * (lane & 1)) : "memory");
#pragma unroll
      for (int g4 = 0; g4 < GP; g4 += 4) {
        const float4 w = *reinterpret_cast<const float4*>(ps + i * GP + g4);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          o[g4][e] = fmaf(w.x, v[e], o[g4][e]);
          o[g4 + 1][e] = fmaf(w.y, v[e], o[g4 + 1][e]);
          o[g4 + 2][e] = fmaf(w.z, v[e], o[g4 + 2][e]);
          o[g4 + 3][e] = fmaf(w.w, v[e], o[g4 + 3][e]);
        }
      }
    }
  }
  __device__ void finish() {
#pragma unroll
    for (int g = 0; g < GP; ++g)
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], s);
  }
  template <class F>
  __device__ void stats(int G, F&& ml) const {
#pragma unroll
    for (int g = 0; g < GP; ++g)
      if ((threadIdx.x & 31) == g && g < G) ml(g, m[g], l[g]);
  }
  __device__ void write(float* to, int G, bool divide) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int g = 0; g < GP; ++g) {
      const float inv = !divide ? 1.f : l[g] > 0.f ? 1.f / l[g] : 0.f;
      if (g < G) {
#pragma unroll
        for (int e = 0; e < E; ++e) to[g * D + lane * E + e] = o[g][e] * inv;
      }
    }
  }
};

// ------------------------------------------------------------- attend
// Shared memory from a 1024-byte boundary; what a warp has, and the line.
template <int D, class M>
struct Plan {
  static constexpr int ES = sizeof(typename M::T);
  static constexpr int SLABS = D * ES / 128;              // 128-byte columns of a row
  static constexpr int ROWS = SLABS * PAGED_GROUP * 128;  // K or V of a group
  static constexpr int STAGE = 2 * ROWS;
  static constexpr int STAGES = 196608 / M::CTAS / (M::WARPS * STAGE);
  static constexpr int OFF_RAW = M::WARPS * STAGES * STAGE;
  static constexpr int OFF_CS = OFF_RAW + M::WARPS * M::RAW;
  static constexpr int OFF_TURNS = OFF_CS + M::WARPS * D / 2 * 8;
  static constexpr int OFF_SCRATCH = OFF_TURNS + D / 2 * 8;
  static constexpr int OFF_BAR = OFF_SCRATCH + M::WARPS * M::SCRATCH;
  static constexpr int OFF_HELD = OFF_BAR + M::WARPS * STAGES * 8;  // whether a stage's page is in the pool
  static constexpr int OFF_SCAN = OFF_HELD + M::WARPS * STAGES * 4;
  static constexpr int OFF_LINE = OFF_SCAN + M::WARPS * 4;
  static constexpr int bytes(int B) { return 1024 + OFF_LINE + (B + 1) * 4; }
  static_assert(bytes(PAGED_MAX_BATCH) <= 232448, "the largest batch fits one CTA");
};

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar,
                                         unsigned long long policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, "
      "%4}], [%5], %6;" ::"r"(dst),
      "l"(map), "r"(0), "r"(row), "r"(0), "r"(bar), "l"(policy)
      : "memory");
}

template <int D, class M>
__global__ void __launch_bounds__(32 * M::WARPS, M::CTAS)
    paged_attend_kernel(const __grid_constant__ PagedAttendParams p, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
  using P = Plan<D, M>;
  constexpr int S = P::STAGES;
  extern __shared__ __align__(16) char raw[];
  char* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.G;
  float2* cs = reinterpret_cast<float2*>(sm + P::OFF_CS) + warp * (D / 2);
  unsigned long long* turns = reinterpret_cast<unsigned long long*>(sm + P::OFF_TURNS);
  float* scratch = reinterpret_cast<float*>(sm + P::OFF_SCRATCH + warp * M::SCRATCH);
  char* query = M::RAW ? sm + P::OFF_RAW + warp * M::RAW : reinterpret_cast<char*>(scratch);
  int* held = reinterpret_cast<int*>(sm + P::OFF_HELD) + warp * S;
  unsigned* words = reinterpret_cast<unsigned*>(sm + P::OFF_LINE);
  const uint32_t ring = smem_u32(sm) + warp * S * P::STAGE;
  const uint32_t bars = smem_u32(sm + P::OFF_BAR) + warp * S * 8;
  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(bars + 8 * i, 1);
    fence_mbar_init();
  }
  // (lanes reading different parameter words take turns: a few lanes of each warp)
  constexpr int TW = D / 2 / M::WARPS;
  if (lane < TW) turns[warp * TW + lane] = p.rope_turns[warp * TW + lane];
  paged_wait();
  fence_proxy_async_global();  // (a kernel before this one may have stored the rows that TMA reads)
  paged_go();  // the join's blocks take their places beside this kernel's, and read the lengths
  make_line<32 * M::WARPS>(p, words, reinterpret_cast<int*>(sm + P::OFF_SCAN), blockIdx.x == 0);
  const PagedLine line{words, p.B, p.Hkv};
  for (int b = blockIdx.x; b < p.B; b += gridDim.x)  // sequences without a token: zeros
    if (line.groups(b) == 0)
      for (int i = tid; i < p.Hq * D; i += 32 * M::WARPS) p.out[(size_t)b * p.Hq * D + i] = 0.f;
  // few parts lie on as many SMs
  const PagedCuts cuts = line.cuts(p.parts);
  const int c = warp * gridDim.x + blockIdx.x;
  if (c >= cuts.n) return;
  const int edge = line.part_begin(cuts, c + (lane & 1));  // both at once
  const int r0 = __shfl_sync(0xffffffffu, edge, 0), r1 = __shfl_sync(0xffffffffu, edge, 1);
  if (r0 == r1) return;

  // K and V are read once: they make way in L2 for what the join reads again (32K
  // tokens 27.4 us without, 26.2 with; one token of eight 4K caches 40.4 and 36.5);
  // a stream of many times L2 with no logits runs up to 1% faster as it comes (2.38 GB:
  // 349.4 us against 353.1)
  unsigned long long policy;
  if (p.weight || (long long)line.total() * P::STAGE < (512ll << 20))
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  else
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
  // The logits stay in L2 as far as they can, and the join drops them there once it
  // has read them: neither K and V push them out nor do they go to memory after use
  // (four sequences of 128K, 67 MB of logits: 352 us, 364 stored as they come, 374
  // without the drop; eight of 4K 28.4, 28.5, 28.1)
  Logits logits;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(logits.policy));
  // Lane i holds the pool row of group (batch of 32) + i of this part.
  const int mine = r1 - r0;
  int rows = -1, issued = 0, landed = 0;
  bool dead = false;  // a wait ran out: nothing more is copied or waited for
  auto look_up = [&](int k) {
    const int x = r0 + k + lane;
    rows = -1;
    if (x < r1) {
      const int b = line.sequence_of(x);
      const int n = line.groups(b), rem = x - line.before(b) * p.Hkv;
      const int h = rem / n, slot = (rem - h * n) * PAGED_GROUP;
      const int page = p.page_table[(size_t)b * p.max_pages + (slot >> p.log2_page)];
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
      const uint32_t bar = bars + 8 * st, dst = ring + st * P::STAGE;
      if (row >= 0) {
        mbar_arrive_expect_tx(bar, P::STAGE);
        if (issued != p.drop_group || c != 0) {  // (test hook: copies that never come)
          tma_rows(dst, &kmap, row, bar, policy);
          tma_rows(dst + P::ROWS, &vmap, row, bar, policy);
        }
      } else {
        mbar_arrive(bar);
      }
    }
    ++issued;
  };
  for (int i = 0; i < S; ++i) issue();

  auto fetch = [&](int unit) {  // a unit's raw query rows
    const char* q = static_cast<const char*>(p.q) + (size_t)unit * G * D * P::ES;
    for (int i = lane; i < G * D * P::ES / 16; i += 32) cp_async16(smem_u32(query) + 16 * i, q + 16 * i);
    cp_async_commit();
  };
  PagedSegments sg;
  sg.start(line, r0, r1);
  sg.at();
  if (M::RAW) fetch(sg.unit());
  int k = 0, turned = -1, pos = p.pos[sg.b];
  for (bool more = true; more;) {
    const int unit = sg.unit(), len = line.tokens(sg.b);
    if (!M::RAW) fetch(unit);
    if (sg.b != turned) {
      turned = sg.b;
      for (int f = lane; f < D / 2; f += 32) {
        const float2 a = rope_cos_sin(turns[f], pos);
        cs[f] = make_float2(a.x * p.scale, a.y * p.scale);
      }
    }
    cp_async_wait<0>();
    __syncwarp();
    M mt;
    mt.begin(query, cs, G, scratch);
    __syncwarp();
    const int first = sg.x, begin = sg.unit_begin, end = sg.unit_end, last = sg.seg_end();
    sg.next();
    more = sg.at();
    if (more) {
      if (M::RAW) fetch(sg.unit());
      pos = p.pos[sg.b];
    }
    logits.to = p.weight ? p.logits + ((size_t)unit * p.T_cap + (size_t)(r0 + k - begin) * PAGED_GROUP) * G : nullptr;
    for (; r0 + k < last; ++k) {
      const int t0 = (r0 + k - begin) * PAGED_GROUP;
      const int st = k % S;
      const uint32_t kb = ring + st * P::STAGE, vb = kb + P::ROWS;
      if (!dead && !mbar_wait_bounded(bars + 8 * st, (k / S) & 1, p.wait_ns)) {
        if (lane == 0) atomicOr(p.status, 2);
        dead = true;
      }
      dead = __any_sync(0xffffffffu, dead);
      if (!dead) landed = k + 1;
      __syncwarp();
      const int n = held[st] && !dead ? min(PAGED_GROUP, len - t0) : 0;
      if (n < PAGED_GROUP) {  // V rows behind the end count for nothing, NaN neither
        for (int i = lane; i < (PAGED_GROUP - n) * P::SLABS * 8; i += 32) {
          const int r = n + i / (P::SLABS * 8), ch = i % (P::SLABS * 8);
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vb + (ch >> 3) * (PAGED_GROUP * 128) + r * 128 +
                                                                        ((ch & 7) << 4)),
                       "r"(0)
                       : "memory");
        }
        fence_proxy_async();
        __syncwarp();
      }
      mt.step(kb, vb, n, logits, G, scratch);
      if (logits.to) logits.to += PAGED_GROUP * G;
      __syncwarp();
      issue();
    }
    mt.finish();
    if (first == begin && last == end) {
      mt.write(p.out + (size_t)unit * G * D, G, true);
      if (p.weight)
        mt.stats(G, [&](int g, float m, float l) { p.lse[(size_t)unit * G + g] = l > 0.f ? m + log2f(l) : INFINITY; });
    } else {
      float* rec = p.records + (size_t)(2 * c + (begin < r0 ? 0 : 1)) * paged_record_floats(G, D);
      mt.write(rec, G, false);
      mt.stats(G, [&](int g, float m, float l) {
        rec[G * D + g] = m;
        rec[G * D + G + g] = l;
      });
    }
  }
  // after a wait that ran out: no copy may land in memory of a block that is gone
  for (; landed < issued; ++landed)
    if (!mbar_wait_bounded(bars + 8 * (landed % S), (landed / S) & 1, 8 * p.wait_ns) && lane == 0) atomicOr(p.status, 4);
}

// --------------------------------------------------------------- join
__device__ __forceinline__ float finite_or_0(float m) { return m == -INFINITY ? 0.f : m; }

// log2 of the softmax denominators over the parts c0 .. c1 of a unit, a whole warp:
// head lane % 8's, four lanes to a head.
__device__ float joined_lse(const PagedAttendParams& p, int R, int GD, int c0, int c1) {
  static_assert(G_MAX == 8, "the lanes of a head");
  const int lane = threadIdx.x & 31, g = min(lane & 7, p.G - 1);
  float M = -INFINITY, L = 0.f;
#pragma unroll 4
  for (int k = c0 + (lane >> 3); k <= c1; k += 4) {
    const float* r = p.records + (size_t)(2 * k + (k == c0)) * R + GD + g;
    const float m = ld_cg(r), l = ld_cg(r + p.G), X = fmaxf(M, m), Xs = finite_or_0(X);
    L = L * exp2f(M - Xs) + l * exp2f(m - Xs);
    M = X;
  }
#pragma unroll
  for (int s = 16; s >= 8; s >>= 1) {
    const float m = __shfl_xor_sync(0xffffffffu, M, s), l = __shfl_xor_sync(0xffffffffu, L, s);
    const float X = fmaxf(M, m), Xs = finite_or_0(X);
    L = L * exp2f(M - Xs) + l * exp2f(m - Xs);
    M = X;
  }
  return L > 0.f ? M + log2f(L) : INFINITY;
}

// Tasks: a slice of the output of a unit that was cut; a task goes by its unit,
// or, where there are more units than parts, by the part the unit begins in.
// Rows of lanes take the unit's records in turn, a lane four floats of each,
// then the rows' sums meet in order.  A warp takes a task (128 floats, its own
// row), or where a unit's parts are many a block does, with its warps as rows, or
// four rows of 8 lanes to a warp (32 floats).
// With weights (GM: the heads that fit the registers, 0 without), each warp then adds
// what its share of the line's tokens gets, by itself; where the tasks take a quarter
// of the warps or less the others do that meanwhile (16 sequences of 500 tokens, 21%:
// 16.7 us, 19.9 with a share for all; 64 of them, 42%: 32.0 and 26.7).  What of a warp's
// share depends on the lengths alone is worked out before the wait (1K tokens: 9.0 us
// against 8.2).
// A block is small enough to wait for the first kernel beside its CTAs.
// With weights a block takes a task where a unit has more parts than this: 8 units of
// 4K tokens, 76 parts each, 12.3 us against 15.9 by warps; 64 of 4K, 9 parts each, 29.4
// against 28.6; 16 of 64K, 38 parts each, 93.1 against 91.0.  (Without weights, where
// nothing else fills the warps, while there are less than two tasks to a block.)
constexpr int JN_MANY = 40;
template <int D, int GM>
__global__ void __launch_bounds__(JN_NT, GM ? 2 : 3)
    paged_join_kernel(const __grid_constant__ PagedAttendParams p) {
  constexpr int NT = JN_NT, NW = NT / 32;
  constexpr bool WEIGHTS = GM > 0;
  extern __shared__ unsigned words[];
  __shared__ float4 so[NT];
  __shared__ float2 sml[NT];
  __shared__ float lse[NW][G_MAX];
  __shared__ int scan[NW];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = p.G;
  const int R = paged_record_floats(G, D);
  // (the lengths are older than the first kernel, which waited before it let this one
  // begin: they are in L2 by then)
  make_line<NT>(p, words, scan, false);
  const PagedLine line{words, p.B, p.Hkv};
  const PagedCuts cuts = line.cuts(p.parts);
  const int parts = cuts.n, total = line.total();
  const int units = p.B * p.Hkv, blocks = gridDim.x;
  const bool by_unit = units <= parts;
  const int most = (by_unit ? units : max(parts - 1, 0)) * ((G * D + 127) / 128);
  const bool team = WEIGHTS ? by_unit && parts > JN_MANY * units : most < 2 * blocks;
  const bool fine = !WEIGHTS && team && by_unit && units * (G * D / 32) <= blocks;
  const int lanes = fine ? 8 : 32, width = 4 * lanes, slices = (G * D + width - 1) / width;
  const int tasks = (by_unit ? units : max(parts - 1, 0)) * slices;
  const int nrows = team ? NT / lanes : 1, row = team ? tid / lanes : 0, at = tid & (lanes - 1);
  // The unit of a task and its parts; false when it was not cut, or does not begin there.
  PagedSegments sg;
  int c0 = 0, c1 = 0;
  auto task_at = [&](int task) {
    const int of = task / slices;
    if (by_unit) {
      const int b = of / p.Hkv, h = of - b * p.Hkv, n = line.groups(b);
      if (n == 0) return false;
      sg.line = line;
      sg.end = total;
      sg.b = b;
      sg.h = h;
      sg.x = line.before(b) * p.Hkv + h * n;
      sg.at();
    } else {
      const int edge = line.part_begin(cuts, of + 1);
      if (edge <= 0 || edge >= total) return false;
      sg.start(line, edge - 1, edge);
      sg.at();
      if (sg.unit_end <= edge) return false;
    }
    c0 = sg.first_part(cuts);
    c1 = sg.last_part(cuts);
    return by_unit ? c0 < c1 : c0 == of;
  };
  const int step = team ? blocks : blocks * NW;
  int task = team ? blockIdx.x : warp * blocks + blockIdx.x;
  bool cut_here = task < tasks && task_at(task);
  // the warps that add weights, and this one's share of the line
  int warps = blocks * NW, w = blockIdx.x * NW + warp;
  if (WEIGHTS && 4 * tasks <= (team ? blocks : warps)) {
    w = team ? w - tasks * NW : warp * blocks + blockIdx.x - tasks;
    warps -= team ? tasks * NW : tasks;
  }
  PagedSegments share;
  int s0 = 0, s1 = 0;  // the parts of its unit
  bool more = WEIGHTS && w >= 0;
  if (more) {
    share.start(line, cut(total, warps, w), cut(total, warps, w + 1));
    more = share.at();
    if (more) {
      s0 = share.first_part(cuts);
      s1 = share.last_part(cuts);
    }
  }
  paged_go();
  paged_wait();
  for (; task < tasks; task += step, cut_here = task < tasks && task_at(task)) {
    if (!cut_here) continue;
    const int n = c1 - c0 + 1;
    const int i0 = (task % slices) * width + 4 * at, i = min(i0, G * D - 4), g = i / D;
    const float* first = p.records + (size_t)(2 * c0 + 1) * R;
    const float* rest = p.records + (size_t)(2 * c0) * R;
    float M = -INFINITY, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 5;
    for (int k0 = row; k0 < n; k0 += U * nrows) {
      float4 o[U];
      float m[U], l[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * nrows;
        const float* r = k == 0 ? first : rest + (size_t)(2 * k) * R;
        o[u] = k < n ? ld_cg(reinterpret_cast<const float4*>(r + i)) : make_float4(0.f, 0.f, 0.f, 0.f);
        m[u] = k < n ? ld_cg(r + G * D + g) : -INFINITY;
        l[u] = k < n ? ld_cg(r + G * D + G + g) : 0.f;
      }
      float X = M;
#pragma unroll
      for (int u = 0; u < U; ++u) X = fmaxf(X, m[u]);
      const float Xs = finite_or_0(X), f = exp2f(M - Xs);
      M = X;
      L *= f;
      a = make_float4(a.x * f, a.y * f, a.z * f, a.w * f);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float e = exp2f(m[u] - Xs);
        L += l[u] * e;
        a = make_float4(a.x + o[u].x * e, a.y + o[u].y * e, a.z + o[u].z * e, a.w + o[u].w * e);
      }
    }
    if (team) {
      for (int s = lanes; s < 32; s <<= 1) {  // the rows of a warp
        const float m = __shfl_xor_sync(0xffffffffu, M, s), X = fmaxf(M, m), Xs = finite_or_0(X);
        const float e = exp2f(M - Xs);
        M = X;
        L *= e;
        a = make_float4(a.x * e, a.y * e, a.z * e, a.w * e);
        L += __shfl_xor_sync(0xffffffffu, L, s);
        a.x += __shfl_xor_sync(0xffffffffu, a.x, s);
        a.y += __shfl_xor_sync(0xffffffffu, a.y, s);
        a.z += __shfl_xor_sync(0xffffffffu, a.z, s);
        a.w += __shfl_xor_sync(0xffffffffu, a.w, s);
      }
      __syncthreads();  // the last task's sums are read
      so[tid] = a;
      sml[tid] = make_float2(M, L);
      __syncthreads();
      if (row == 0) {
        float X = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) X = fmaxf(X, sml[w * 32 + lane].x);
        const float Xs = finite_or_0(X);
        L = 0.f;
        a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float2 s = sml[w * 32 + lane];
          const float e = exp2f(s.x - Xs);
          const float4 o = so[w * 32 + lane];
          L += s.y * e;
          a = make_float4(a.x + o.x * e, a.y + o.y * e, a.z + o.z * e, a.w + o.w * e);
        }
      }
    }
    if (row == 0 && i0 < G * D) {
      const float inv = L > 0.f ? 1.f / L : 0.f;
      *reinterpret_cast<float4*>(p.out + (size_t)sg.unit() * G * D + i) =
          make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    }
  }
  if constexpr (WEIGHTS) while (more) {
    const int unit = share.unit();
    // four tokens a lane: a group's slots, and so its logits and weights, are all
    // there (those behind the end are -inf and get nothing); the first are under way
    // while the parts' sums are joined
    const int t0 = (share.x - share.unit_begin) * PAGED_GROUP, t1 = (share.seg_end() - share.unit_begin) * PAGED_GROUP;
    const int tokens = line.tokens(share.b);
    const float* z = p.logits + (size_t)unit * G * p.T_cap;
    float* weight = p.weight + (size_t)unit * p.T_cap;
    float4 zg[GM], old;
    auto load = [&](int t) {
      const float* zt = z + (size_t)(t & -PAGED_GROUP) * G + (t & (PAGED_GROUP - 1));
#pragma unroll
      for (int g = 0; g < GM; ++g)
        if (g < G) zg[g] = ld_cg(reinterpret_cast<const float4*>(zt + g * PAGED_GROUP));
      old = *reinterpret_cast<const float4*>(weight + t);
    };
    int t = t0 + 4 * lane;
    if (t < t1) load(t);
    const float mine = s0 == s1 ? ld_cg(p.lse + (size_t)unit * G + min(lane, G - 1)) : joined_lse(p, R, G * D, s0, s1);
    __syncwarp();  // (the last unit's are read)
    if (lane < G) lse[warp][lane] = mine;
    __syncwarp();
    while (t < t1) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int g = 0; g < GM; ++g)
        if (g < G) {
          const float e = lse[warp][g];
          a.x += exp2f(zg[g].x - e);
          a.y += exp2f(zg[g].y - e);
          a.z += exp2f(zg[g].z - e);
          a.w += exp2f(zg[g].w - e);
        }
      const int live = tokens - t;  // slots behind the end keep what they hold
      if (live >= 4) {
        *reinterpret_cast<float4*>(weight + t) = make_float4(old.x + a.x, old.y + a.y, old.z + a.z, old.w + a.w);
      } else {
        if (live > 0) weight[t] = old.x + a.x;
        if (live > 1) weight[t + 1] = old.y + a.y;
        if (live > 2) weight[t + 2] = old.z + a.z;
      }
      t += 4 * 32;
      if (t < t1) load(t);
    }
    __syncwarp();
    // the whole lines of logits that only this warp read
    const uintptr_t z0 = reinterpret_cast<uintptr_t>(z + (size_t)t0 * G);
    const uintptr_t z1 = reinterpret_cast<uintptr_t>(z + (size_t)t1 * G) & ~(uintptr_t)127;
    for (uintptr_t at = ((z0 + 127) & ~(uintptr_t)127) + 128 * lane; at < z1; at += 128 * 32)
      asm volatile("discard.global.L2 [%0], 128;" ::"l"(at) : "memory");
    share.next();
    more = share.at();
    if (more) {
      s0 = share.first_part(cuts);
      s1 = share.last_part(cuts);
    }
  }
}

// -------------------------------------------------------------- launch
// A pool of pages as rows of 128-byte slabs: a copy takes a group's 16 rows.
cudaError_t pool_map(CUtensorMap* map, const void* pool, long long rows, int D, int es, CUtensorMapDataType type) {
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
  const int cols = 128 / es;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)(D / cols)};
  const cuuint64_t strides[2] = {(cuuint64_t)D * es, 128};
  const cuuint32_t box[3] = {(cuuint32_t)cols, PAGED_GROUP, (cuuint32_t)(D / cols)}, one[3] = {1, 1, 1};
  const CUresult r = encode(map, type, 3, const_cast<void*>(pool), dims, strides, box, one,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The kernel's shared memory, for the largest batch, once a device.
template <int D, class M>
cudaError_t allow_shared() {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(paged_attend_kernel<D, M>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Plan<D, M>::bytes(PAGED_MAX_BATCH));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

template <int D, class M>
cudaError_t launch(PagedAttendParams& p, int sms, cudaStream_t s) {
  CUtensorMap km, vm;
  const long long rows = ((long long)p.n_pages * p.Hkv) << p.log2_page;
  cudaError_t e = pool_map(&km, p.k_pages, rows, D, sizeof(typename M::T), M::TYPE);
  if (e == cudaSuccess) e = pool_map(&vm, p.v_pages, rows, D, sizeof(typename M::T), M::TYPE);
  if (e != cudaSuccess) return e;
  const int smem = Plan<D, M>::bytes(p.B);
  // as many parts as warps are resident at once: M::CTAS CTAs to an SM while the
  // lengths of the batch leave them the room (228 KB, 1 KB of it each CTA's system's)
  const int ctas = M::CTAS * (smem + 1024) <= 233472 ? M::CTAS : 1;
  const int grid = min(ctas * sms, PAGED_MAX_PARTS / M::WARPS);
  p.parts = grid * M::WARPS;
  e = allow_shared<D, M>();
  if (e != cudaSuccess) return e;
  e = paged_behind(paged_attend_kernel<D, M>, grid, 32 * M::WARPS, smem, 0, s, p, km, vm);
  if (e != cudaSuccess) return e;
  const size_t line = (p.B + 1) * 4;
  if (!p.weight) return paged_behind(paged_join_kernel<D, 0>, sms, JN_NT, line, 0, s, p);
  return paged_behind(p.G <= 4 ? paged_join_kernel<D, 4> : paged_join_kernel<D, 8>, 2 * sms, JN_NT, line, 0, s, p);
}

}  // namespace

cudaError_t launch_paged_attend(const PagedAttendParams& p0, int head_dim, bool bf16, int sms, cudaStream_t s) {
  PagedAttendParams p = p0;
  if (bf16 && head_dim == 128)
    return p.G <= 4 ? launch<128, MathBf16<128, true>>(p, sms, s) : launch<128, MathBf16<128, false>>(p, sms, s);
  if (bf16) return p.G <= 4 ? launch<64, MathBf16<64, true>>(p, sms, s) : launch<64, MathBf16<64, false>>(p, sms, s);
  if (head_dim == 128) return p.G <= 4 ? launch<128, MathF32<128, 4>>(p, sms, s) : launch<128, MathF32<128, 8>>(p, sms, s);
  return p.G <= 4 ? launch<64, MathF32<64, 4>>(p, sms, s) : launch<64, MathF32<64, 8>>(p, sms, s);
}

}  // namespace fasa
