// New tokens on their way to the paged cache: their pages, slots and positions
// (assign), then their queries, keys and values (rope_append).
#include <cuda_bf16.h>
#include <stdint.h>

#include "fasa_cluster.cuh"
#include "fasa_internal.h"
#include "fasa_ptx.cuh"
#include "fasa_serve.h"

namespace fasa {
namespace {

// ------------------------------------------------------------------- assign
// Three prefix sums over the sequences (pages given back, pages taken, tokens) say
// everything: the first growing sequence that does not fit, by the sums through it, ends
// the service, and a new token finds its sequence in the tokens' sums, its page in the
// table or, by the pages' sums, in the list.  Every block makes the sums for itself and
// takes its share of the map, so no block waits for another: places of the list below
// free_count are only read, those behind it only written, and a page that is given back
// and taken in the same call is read from the table, whose entries are either given back
// (and stay) or new.
constexpr int AS_NT = 1024;
constexpr int AS_RUN = PAGED_MAX_BATCH / AS_NT;  // sequences of a thread

struct AssignShared {
  int gives[PAGED_MAX_BATCH + 1], takes[PAGED_MAX_BATCH + 1], tokens[PAGED_MAX_BATCH + 1];  // sums before b
  int have[PAGED_MAX_BATCH], want[PAGED_MAX_BATCH];
  int3 scan[AS_NT / 32];
  int first_refused;
};

// The last b of 0 .. B-1 with sum[b] <= x.
__device__ __forceinline__ int sequence_at(const int* sum, int B, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sum[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// What a call comes to: the sums in `sh`, of the sequences that are served.
struct Assignment {
  int n, avail, taken, tokens, r;  // free entries before and with what comes back; r: the first refused (B: none)
};

__device__ Assignment assignment(const AssignParams& p, AssignShared& sh, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ps = (1 << p.log2_page) - 1;
  auto pages = [&](int t) { return (t + ps) >> p.log2_page; };
  auto cap = [&](int t) { return min(max(t, 0), p.T_cap); };
  if (tid == 0) sh.first_refused = p.B;
  bool bad = false;
  int3 x[AS_RUN], sum = make_int3(0, 0, 0);
#pragma unroll
  for (int i = 0; i < AS_RUN; ++i) {
    const int b = AS_RUN * tid + i;
    x[i] = make_int3(0, 0, 0);
    if (b < p.B) {
      const int h0 = p.have[b], w0 = p.want[b], h = cap(h0), w = cap(w0);
      bad = bad || h != h0 || w != w0;
      sh.have[b] = h;
      sh.want[b] = w;
      x[i] = make_int3(max(pages(h) - pages(w), 0), max(pages(w) - pages(h), 0), max(w - h, 0));
    }
    sum.x += x[i].x;
    sum.y += x[i].y;
    sum.z += x[i].z;
  }
  const int n0 = p.free_count[0], n = min(max(n0, 0), p.n_pages);
  bad = bad || n != n0;
  int3 incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, incl.x, o), b = __shfl_up_sync(0xffffffffu, incl.y, o),
              c = __shfl_up_sync(0xffffffffu, incl.z, o);
    if (lane >= o) {
      incl.x += a;
      incl.y += b;
      incl.z += c;
    }
  }
  if (lane == 31) sh.scan[warp] = incl;
  __syncthreads();
  int3 before = make_int3(incl.x - sum.x, incl.y - sum.y, incl.z - sum.z);
  int freed = 0;
#pragma unroll
  for (int v = 0; v < AS_NT / 32; ++v) {
    const int3 s = sh.scan[v];
    freed += s.x;
    if (v < warp) {
      before.x += s.x;
      before.y += s.y;
      before.z += s.z;
    }
  }
  const int avail = (int)min((long long)n + freed, (long long)p.n_pages);
  if ((long long)n + freed > p.n_pages) bad = true;
#pragma unroll
  for (int i = 0; i < AS_RUN; ++i) {
    const int b = AS_RUN * tid + i;
    if (b <= p.B) {
      sh.gives[b] = before.x;
      sh.takes[b] = before.y;
      sh.tokens[b] = before.z;
    }
    before.x += x[i].x;
    before.y += x[i].y;
    before.z += x[i].z;
    if (x[i].z > 0 && (before.y > avail || before.z > p.max_tokens)) atomicMin(&sh.first_refused, b);
  }
  if (tid == AS_NT - 1 && p.B == PAGED_MAX_BATCH) {
    sh.gives[p.B] = before.x;
    sh.takes[p.B] = before.y;
    sh.tokens[p.B] = before.z;
  }
  if (report && bad) atomicOr(p.status, 1);
  __syncthreads();
  const int r = sh.first_refused;
  return Assignment{n, avail, sh.takes[r], sh.tokens[r], r};
}

__device__ void map_tokens(const AssignParams& p, const AssignShared& sh, const Assignment& a) {
  const int ps = (1 << p.log2_page) - 1;
  bool bad = false;
  const int start = blockIdx.x * AS_NT + threadIdx.x, step = gridDim.x * AS_NT;
  for (int x = start; x < p.max_tokens; x += step) {
    int4 m = make_int4(-1, -1, -1, -1);
    if (x < a.tokens) {
      const int b = sequence_at(sh.tokens, p.B, x), j = x - sh.tokens[b];
      const int slot = sh.have[b] + j, e = slot >> p.log2_page;
      const int nth = e - ((sh.have[b] + ps) >> p.log2_page);  // of its new pages
      int* entry = p.page_table + (size_t)b * p.max_pages + e;
      int page;
      if (nth < 0) {
        page = *entry;
      } else {
        const int at = a.avail - 1 - (sh.takes[b] + nth);  // in the list
        if (at < a.n) {
          page = p.free_pages[at];
        } else {  // one that this call gets back
          const int from = sequence_at(sh.gives, p.B, at - a.n);
          const int old = ((sh.want[from] + ps) >> p.log2_page) + (at - a.n - sh.gives[from]);
          page = p.page_table[(size_t)from * p.max_pages + old];
        }
        bad = bad || page < 0 || page >= p.n_pages;
        if ((slot & ps) == 0) *entry = page;
      }
      m = make_int4(b, slot, page, (p.pos ? p.pos[b] : sh.have[b]) + j);
    }
    p.token_map[x] = m;
  }
  // what comes back, behind the list's end
  for (int y = start; y < sh.gives[p.B]; y += step) {
    const int from = sequence_at(sh.gives, p.B, y);
    const int page = p.page_table[(size_t)from * p.max_pages + ((sh.want[from] + ps) >> p.log2_page) + (y - sh.gives[from])];
    bad = bad || page < 0 || page >= p.n_pages;
    if (a.n + y < p.n_pages) p.free_pages[a.n + y] = page;
  }
  if (bad) atomicOr(p.status, 1);
}

__device__ void write_lens(const AssignParams& p, const AssignShared& sh, const Assignment& a) {
  for (int b = threadIdx.x; b <= p.B; b += AS_NT) {
    p.cu_new[b] = sh.tokens[min(b, a.r)];
    if (b < p.B) p.lens_out[b] = b >= a.r && sh.want[b] > sh.have[b] ? sh.have[b] : sh.want[b];
  }
  if (threadIdx.x == 0) p.free_count_out[0] = a.avail - a.taken;
}

// MAP, LENS: what this launch writes.  The lengths may be written where they were read,
// so that they wait for every block: one, where a thread takes a token at most, a cluster,
// or a launch of their own behind as many as there is work for.  64, 1024, 4096, 12.8K,
// 25.6K, 64K and 256K tokens: 3.5, 4.0, 7.3, 12.8, 22.0, 49 and 186 us by one block, 3.9,
// 4.3, 4.6, 5.1, 6.9, 10.7 and 28 by a cluster of eight, 5.8, 6.3, 6.5, 6.2, 6.3, 7.9 and
// 8.7 by two launches.
constexpr int AS_CLUSTER_TOKENS = 16384;
template <bool MAP, bool LENS>
__global__ void __launch_bounds__(AS_NT) paged_assign_kernel(const AssignParams p) {
  __shared__ AssignShared sh;
  paged_go();
  paged_wait();
  const Assignment a = assignment(p, sh, MAP && blockIdx.x == 0);
  if (MAP) map_tokens(p, sh, a);
  if (MAP && LENS) {
    if (cluster_size() > 1) cluster_sync();
    else __syncthreads();
  }
  if (LENS && blockIdx.x == 0) write_lens(p, sh, a);
}

// -------------------------------------------------------------- rope_append
// A warp takes a token and some of its rows (query heads, key heads, value heads), two
// 16-byte chunks of a row to a lane: chunk i of the turned part and chunk i + half of it
// (or, behind it, two neighbours), so that a lane holds both elements of its pairs in
// either layout, and the same ones in every head: their cosines are worked out once.
constexpr int RA_NT = 128;
constexpr int RA_U = 2;  // rows that a lane has on the way
// Warps of a launch for an SM, about: a warp takes as many rows of its token as that leaves
// it.  40 heads of 128 dims and 8 of values, 32, 512, 2048 and 4096 tokens: 4 rows to a warp
// 2.1, 4.8, 12.6 and 25.4 us, 8 rows 2.2, 3.7, 8.8 and 17.2, 24 rows 3.7, 5.7, 6.7 and 16.2,
// all 48 rows 5.7, 6.9, 10.3 and 15.3.
constexpr int RA_WARPS = 27;

// Element e of a chunk in fp32, and back.
template <typename T>
__device__ __forceinline__ float element(const uint4& w, int e) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  if constexpr (sizeof(T) == 2) return e & 1 ? bf16_hi(u[e >> 1]) : bf16_lo(u[e >> 1]);
  else return __uint_as_float(u[e]);
}
template <typename T>
__device__ __forceinline__ uint4 chunk_of(const float (&x)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 2)
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  else
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

template <typename T, int D, bool HALF>
__global__ void __launch_bounds__(RA_NT) rope_append_kernel(const __grid_constant__ RopeAppendParams p, int rows_each) {
  constexpr int EPC = 16 / (int)sizeof(T);                       // elements of a chunk
  constexpr int LPR = D / EPC / 2, RPW = 32 / LPR;               // lanes of a row, rows of a warp
  constexpr int TW = D / 2 / (RA_NT / 32);
  __shared__ unsigned long long turns[D / 2];
  __shared__ __align__(16) float2 angles[RA_NT / 32][D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // (lanes reading different parameter words take turns: some lanes of each warp)
  if (lane < TW) turns[warp * TW + lane] = p.turns[warp * TW + lane];
  __syncthreads();
  paged_go();
  paged_wait();
  const int nq = p.q ? p.Hq : 0, rows = nq + (p.k ? 2 * p.Hkv : 0);
  const int groups = (rows + rows_each - 1) / rows_each, at = lane % LPR, sub = lane / LPR;
  const int rc = p.rotary_dim / EPC;  // chunks that are turned
  const bool turned = at < rc / 2;
  const int c0 = turned ? at : rc + 2 * (at - rc / 2), c1 = turned ? at + rc / 2 : c0 + 1;
  const long long items = (long long)p.n_tokens * groups, warps = (long long)gridDim.x * (RA_NT / 32);
  for (long long w = (long long)blockIdx.x * (RA_NT / 32) + warp; w < items; w += warps) {
    const int x = (int)(w / groups), r0 = (int)(w - (long long)x * groups) * rows_each, r1 = min(rows, r0 + rows_each);
    // the rows first: they need only x, the rest is a chain of loads
    uint4 a[RA_U], b[RA_U];
    auto load = [&](int rb) {
#pragma unroll
      for (int i = 0; i < RA_U; ++i) {
        const int r = rb + i * RPW + sub;
        if (r < r1) {
          const T* from = r < nq ? static_cast<const T*>(p.q) + x * p.q_stride + (size_t)r * D
                          : r < nq + p.Hkv
                              ? static_cast<const T*>(p.k) + x * p.k_stride + (size_t)(r - nq) * D
                              : static_cast<const T*>(p.v) + x * p.v_stride + (size_t)(r - nq - p.Hkv) * D;
          a[i] = reinterpret_cast<const uint4*>(from)[c0];
          b[i] = reinterpret_cast<const uint4*>(from)[c1];
        }
      }
    };
    load(r0);
    const int4 m = p.token_map[x];  // sequence, slot, page, position
    if (m.x < 0) continue;
    if (m.x >= p.B || m.y < 0 || m.y >= p.T_cap || m.z < 0 || m.z >= p.n_pages) {
      if (lane == 0) atomicOr(p.status, 1);
      continue;
    }
    __syncwarp();  // (the last token's are read)
#pragma unroll 1
    for (int f = lane; f < p.rotary_dim / 2; f += 32) {
      const float2 cs = rope_cos_sin(turns[f], m.w);
      angles[warp][f] = make_float2(cs.x * p.magnitude, cs.y * p.magnitude);
    }
    __syncwarp();
    // HALF: pair e is element e of both chunks; else pairs are neighbours in a chunk
    float2 cs[EPC];
#pragma unroll
    for (int e = 0; e < EPC; ++e) {
      const int f = HALF ? c0 * EPC + e : (e < EPC / 2 ? c0 * (EPC / 2) + e : c1 * (EPC / 2) + e - EPC / 2);
      cs[e] = turned ? angles[warp][f] : make_float2(1.f, 0.f);
    }
    for (int rb = r0; rb < r1; rb += RPW * RA_U) {
      if (rb > r0) load(rb);
#pragma unroll
      for (int i = 0; i < RA_U; ++i) {
        const int r = rb + i * RPW + sub;
        if (r < r1) {
          uint4 ya = a[i], yb = b[i];
          if (turned && r < nq + p.Hkv) {
            float u[EPC], v[EPC];
#pragma unroll
            for (int e = 0; e < EPC; ++e) {
              u[e] = element<T>(a[i], e);
              v[e] = element<T>(b[i], e);
            }
            if constexpr (HALF) {
#pragma unroll
              for (int e = 0; e < EPC; ++e) {
                const float y0 = u[e] * cs[e].x - v[e] * cs[e].y, y1 = u[e] * cs[e].y + v[e] * cs[e].x;
                u[e] = y0;
                v[e] = y1;
              }
            } else {
#pragma unroll
              for (int e = 0; e < EPC / 2; ++e) {
                const float2 s = cs[e], t = cs[e + EPC / 2];
                const float u0 = u[2 * e], u1 = u[2 * e + 1], v0 = v[2 * e], v1 = v[2 * e + 1];
                u[2 * e] = u0 * s.x - u1 * s.y;
                u[2 * e + 1] = u0 * s.y + u1 * s.x;
                v[2 * e] = v0 * t.x - v1 * t.y;
                v[2 * e + 1] = v0 * t.y + v1 * t.x;
              }
            }
            ya = chunk_of<T>(u);
            yb = chunk_of<T>(v);
          }
          const int h = r < nq + p.Hkv ? r - nq : r - nq - p.Hkv;
          T* to = r < nq ? static_cast<T*>(p.q_out) + ((size_t)x * p.Hq + r) * D
                         : static_cast<T*>(r < nq + p.Hkv ? p.k_pages : p.v_pages) +
                               (size_t)paged_row(m.z, p.n_pages, p.Hkv, h, p.log2_page, m.y) * D;
          reinterpret_cast<uint4*>(to)[c0] = ya;
          reinterpret_cast<uint4*>(to)[c1] = yb;
          if (at == 0 && r >= nq && r < nq + p.Hkv) {
            const size_t stat = ((size_t)m.x * p.Hkv + h) * p.T_cap + m.y;
            if (p.weight) p.weight[stat] = 0.f;
            if (p.token_pos) p.token_pos[stat] = m.w;
          }
        }
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch_rope(const RopeAppendParams& p, bool half, int sms, cudaStream_t s) {
  constexpr int RPW = 32 / (D * (int)sizeof(T) / 32);
  const int rows = (p.q ? p.Hq : 0) + (p.k ? 2 * p.Hkv : 0);
  const long long steps = ((long long)p.n_tokens * rows / RPW + RA_WARPS * sms - 1) / (RA_WARPS * sms);
  const int each = (int)(steps * RPW < RPW ? RPW : steps * RPW < rows ? steps * RPW : rows);
  const long long items = (long long)p.n_tokens * ((rows + each - 1) / each), blocks = (items + RA_NT / 32 - 1) / (RA_NT / 32);
  const int grid = (int)(blocks < 16ll * sms ? blocks : 16ll * sms);
  return paged_behind(half ? rope_append_kernel<T, D, true> : rope_append_kernel<T, D, false>, grid, RA_NT, 0, 0, s, p,
                      each);
}

}  // namespace

cudaError_t launch_paged_assign(const AssignParams& p, int sms, cudaStream_t s) {
  if (p.max_tokens <= AS_NT) return paged_behind(paged_assign_kernel<true, true>, 1, AS_NT, 0, 0, s, p);
  if (p.max_tokens <= AS_CLUSTER_TOKENS) return paged_behind(paged_assign_kernel<true, true>, 8, AS_NT, 0, 8, s, p);
  const int blocks = (p.max_tokens + AS_NT - 1) / AS_NT;
  const cudaError_t e = paged_behind(paged_assign_kernel<true, false>, blocks < sms ? blocks : sms, AS_NT, 0, 0, s, p);
  return e != cudaSuccess ? e : paged_behind(paged_assign_kernel<false, true>, 1, AS_NT, 0, 0, s, p);
}

cudaError_t launch_rope_append(const RopeAppendParams& p, int head_dim, bool bf16, bool half, int sms, cudaStream_t s) {
  if (bf16) return head_dim == 128 ? launch_rope<__nv_bfloat16, 128>(p, half, sms, s) : launch_rope<__nv_bfloat16, 64>(p, half, sms, s);
  return head_dim == 128 ? launch_rope<float, 128>(p, half, sms, s) : launch_rope<float, 64>(p, half, sms, s);
}

}  // namespace fasa
