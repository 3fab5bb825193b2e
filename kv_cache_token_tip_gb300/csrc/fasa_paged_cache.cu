// Writing and cutting the paged cache: the append of new tokens and the
// eviction by accumulated attention weight.
#include <cuda_bf16.h>
#include <stdint.h>

#include "fasa_cluster.cuh"
#include "fasa_internal.h"
#include "fasa_paged.h"
#include "fasa_ptx.cuh"

namespace fasa {
namespace {

// ------------------------------------------------------------------- append
constexpr int AP_NT = 128;

// Sequence of new token x, and which of its tokens it is; false for padding
// and for a table that does not ascend (reported).
__device__ __forceinline__ bool token_of(const PagedAppendParams& p, int x, int& b, int& j) {
  if (!p.cu_new) {
    b = x;
    j = 0;
    return true;
  }
  if (x >= __ldg(p.cu_new + p.B)) return false;  // padding
  int lo = 0, hi = p.B;  // cu_new[lo] <= x < cu_new[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu_new + mid) <= x) lo = mid;
    else hi = mid;
  }
  const int first = __ldg(p.cu_new + lo), next = __ldg(p.cu_new + lo + 1);
  b = lo;
  j = x - first;
  if (first < 0 || first > x || next <= x || next > p.n_tokens) {
    atomicOr(p.status, 1);
    return false;
  }
  return true;
}

// One warp per (token, KV head): the key's pairs turned by the token's
// position, the value copied.  Elements of a lane: D / 32, whole pairs.
template <typename T, int D>
__global__ void __launch_bounds__(AP_NT) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = ((long long)blockIdx.x * AP_NT + threadIdx.x) >> 5;
  const int x = (int)(w / p.Hkv), h = (int)(w - (long long)x * p.Hkv);
  if (x >= p.n_tokens) return;
  int b, j;
  if (!token_of(p, x, b, j)) return;
  const int len = p.seq_lens[b];
  const long long slot = (long long)len + j;
  if (len < 0 || slot >= p.T_cap) {
    if (lane == 0) atomicOr(p.status, 1);
    return;
  }
  const int page = p.page_table[(size_t)b * p.max_pages + (slot >> p.log2_page)];
  const long long row = paged_row(page, p.n_pages, p.Hkv, h, p.log2_page, (int)slot);
  if (row < 0) {
    if (lane == 0) atomicOr(p.status, 1);
    return;
  }
  const int m = p.pos[b] + j;
  const T* kn = static_cast<const T*>(p.k_new) + ((size_t)x * p.Hkv + h) * D + lane * E;
  const T* vn = static_cast<const T*>(p.v_new) + ((size_t)x * p.Hkv + h) * D + lane * E;
  T* kd = static_cast<T*>(p.k_pages) + (size_t)row * D + lane * E;
  T* vd = static_cast<T*>(p.v_pages) + (size_t)row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float2 c = rope_cos_sin(p.rope_turns[(lane * E + e) / 2], m);
    const float x0 = to_f32<T>(kn[e]), x1 = to_f32<T>(kn[e + 1]);
    kd[e] = from_f32<T>(x0 * c.x - x1 * c.y);
    kd[e + 1] = from_f32<T>(x0 * c.y + x1 * c.x);
    vd[e] = vn[e];
    vd[e + 1] = vn[e + 1];
  }
  if (lane == 0) {
    const size_t at = ((size_t)b * p.Hkv + h) * p.T_cap + slot;
    if (p.weight) p.weight[at] = 0.f;
    if (p.token_pos) p.token_pos[at] = m;
  }
}

// -------------------------------------------------------------------- evict
constexpr int EV_NT = 1024;
constexpr int EV_NW = EV_NT / 32;
constexpr int EV_BINS = 2048;

struct EvictScratch {
  int scan[EV_NW];
  unsigned mn, mx;
  int bin, above, cnt;
};

// What the selection orders by: held tokens above every weight, NaN below.
__device__ __forceinline__ unsigned evict_key(float w, int tp, int sinks, long long recent_after) {
  if (tp < sinks || (long long)tp > recent_after) return 0xffffffffu;
  return w != w ? 0u : score_key(w);
}

// Exclusive prefix sum over the block (thread order) and the total.
__device__ int block_scan(int x, EvictScratch* sc, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sc->scan[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int v = sc->scan[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    sc->scan[lane] = v;
  }
  __syncthreads();
  total = sc->scan[EV_NW - 1];
  const int before = warp ? sc->scan[warp - 1] : 0;
  __syncthreads();
  return before + incl - x;
}

// One block per (sequence, KV head).
__global__ void __launch_bounds__(EV_NT) paged_evict_kernel(const __grid_constant__ PagedEvictParams p) {
  __shared__ EvictScratch sc;
  __shared__ int hist[EV_BINS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int u = blockIdx.x, b = u / p.Hkv, h = u - b * p.Hkv;
  int len = p.seq_lens[b];
  if (len < 0 || len > p.T_cap) {
    if (tid == 0) atomicOr(p.status, 1);
    len = min(max(len, 0), p.T_cap);
  }
  const int keep = p.keep, left = min(len, keep);
  if (h == 0 && tid == 0) p.new_lens[b] = left;
  const size_t base = (size_t)u * p.T_cap;
  const float* w = p.weight + base;
  const int* tp = p.token_pos + base;
  float* wo = p.weight_out + base;
  int* to = p.token_pos_out + base;
  if (wo != w)  // into other buffers: the holes among these are written over below
    for (int t = tid; t < left; t += EV_NT) {
      wo[t] = w[t];
      to[t] = tp[t];
    }
  if (len <= keep) return;
  const long long after = (long long)p.pos[b] - p.recent;
  auto key_at = [&](int t) { return evict_key(w[t], tp[t], p.sinks, after); };
  // 1. the range of the keys
  if (tid == 0) {
    sc.mn = 0xffffffffu;
    sc.mx = 0u;
  }
  __syncthreads();
  unsigned mn = 0xffffffffu, mx = 0u;
  for (int t = tid; t < len; t += EV_NT) {
    const unsigned k = key_at(t);
    mn = min(mn, k);
    mx = max(mx, k);
  }
  mn = __reduce_min_sync(0xffffffffu, mn);
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (lane == 0) {
    atomicMin(&sc.mn, mn);
    atomicMax(&sc.mx, mx);
  }
  __syncthreads();
  // 2. the bin of the keep-th largest key, narrowed until it is kept whole or
  // is a single key
  unsigned lo = sc.mn, hi = sc.mx, tie_key = 0u;
  unsigned long long from = 0ull;  // keys from here on are kept
  int kr = keep, need = 0;         // and the first `need` slots of tie_key
  while (true) {
    const int shift = max(0, 32 - __clz(hi - lo) - 11);
    for (int i = tid; i < EV_BINS; i += EV_NT) hist[i] = 0;
    __syncthreads();
    for (int t = tid; t < len; t += EV_NT) {
      const unsigned k = key_at(t);
      if (k >= lo && k <= hi) atomicAdd(&hist[(k - lo) >> shift], 1);
    }
    __syncthreads();
    // thread j: bins 2047 - 2j and the one below
    const int hb = EV_BINS - 1 - 2 * tid;
    const int c0 = hist[hb], c1 = hist[hb - 1];
    int tot;
    const int above = block_scan(c0 + c1, &sc, tot);
    if (above < kr && kr <= above + c0 + c1) {
      const bool first = kr <= above + c0;
      sc.bin = first ? hb : hb - 1;
      sc.above = first ? above : above + c0;
      sc.cnt = first ? c0 : c1;
    }
    __syncthreads();
    const int d = sc.bin, cnt = sc.cnt;
    kr -= sc.above;
    __syncthreads();
    const unsigned b0 = lo + ((unsigned)d << shift);
    if (cnt == kr) {
      from = b0;
      break;
    }
    if (shift == 0) {
      tie_key = b0;
      from = (unsigned long long)b0 + 1ull;
      need = kr;
      break;
    }
    hi = b0 + min(hi - b0, (1u << shift) - 1u);  // (b0 + the bin's width may pass 2^32)
    lo = b0;
  }
  // 3. holes and movers in slot order
  int2* moves = p.moves + (size_t)u * p.move_cap;
  int ties = 0, holes = 0, movers = 0;
  for (int t0 = 0; t0 < len; t0 += EV_NT) {
    const int t = t0 + tid;
    const unsigned k = t < len ? key_at(t) : 0u;
    bool kept = t < len && (unsigned long long)k >= from;
    if (need) {
      const bool tie = t < len && k == tie_key;
      int tot;
      const int r = ties + block_scan(tie, &sc, tot);
      if (tie && r < need) kept = true;
      ties += tot;
    }
    const bool hole = t < keep && !kept, mover = kept && t >= keep;
    int tot;
    const int r = block_scan((int)hole | ((int)mover << 16), &sc, tot);
    if (hole) moves[holes + (r & 0xffff)].x = t;
    if (mover) moves[movers + (r >> 16)].y = t;
    holes += tot & 0xffff;
    movers += tot >> 16;
  }
  __syncthreads();
  // 4. the moves, one warp each
  const int n16 = p.row_bytes / 16;
  for (int i = warp; i < holes; i += EV_NW) {
    const int2 mv = moves[i];
    const int* table = p.page_table + (size_t)b * p.max_pages;
    const long long rd = paged_row(table[mv.x >> p.log2_page], p.n_pages, p.Hkv, h, p.log2_page, mv.x);
    const long long rs = paged_row(table[mv.y >> p.log2_page], p.n_pages, p.Hkv, h, p.log2_page, mv.y);
    if (lane == 0) {
      wo[mv.x] = w[mv.y];
      to[mv.x] = tp[mv.y];
    }
    if (rd < 0 || rs < 0) {
      if (lane == 0) atomicOr(p.status, 1);
      continue;
    }
    uint4* kd = reinterpret_cast<uint4*>(static_cast<char*>(p.k_pages) + rd * p.row_bytes);
    const uint4* ks = reinterpret_cast<const uint4*>(static_cast<const char*>(p.k_pages) + rs * p.row_bytes);
    uint4* vd = reinterpret_cast<uint4*>(static_cast<char*>(p.v_pages) + rd * p.row_bytes);
    const uint4* vs = reinterpret_cast<const uint4*>(static_cast<const char*>(p.v_pages) + rs * p.row_bytes);
    for (int c = lane; c < 2 * n16; c += 32) {
      if (c < n16) kd[c] = ks[c];
      else vd[c - n16] = vs[c - n16];
    }
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, int head_dim, bool bf16, cudaStream_t s) {
  const long long warps = (long long)p.n_tokens * p.Hkv;
  const unsigned blocks = (unsigned)((warps * 32 + AP_NT - 1) / AP_NT);
  using B16 = __nv_bfloat16;
  if (bf16) {
    if (head_dim == 128) paged_append_kernel<B16, 128><<<blocks, AP_NT, 0, s>>>(p);
    else paged_append_kernel<B16, 64><<<blocks, AP_NT, 0, s>>>(p);
  } else {
    if (head_dim == 128) paged_append_kernel<float, 128><<<blocks, AP_NT, 0, s>>>(p);
    else paged_append_kernel<float, 64><<<blocks, AP_NT, 0, s>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_paged_evict(const PagedEvictParams& p, cudaStream_t s) {
  paged_evict_kernel<<<p.B * p.Hkv, EV_NT, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace fasa
