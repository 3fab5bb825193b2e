// What the kernels of the attention of chunks share: the line of units in shared
// memory, the join of units that were cut, and the units of the weights' pass.
//
// For a row (a new token and a query head) with z_t = log2(e) q . K_t / sqrt(d) over the
// slots that the token sees: m = max z_t, l = sum 2^(z_t - m), o = sum 2^(z_t - m) V_t,
// out = o / l.  Two parts (m, l, o), (m', l', o') of a row join as M = max(m, m'),
// l 2^(m - M) + l' 2^(m' - M), and o alike.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <mutex>

#include "fasa_ptx.cuh"
#include "fasa_serve.h"

namespace fasa {

// The line, its costs in `before` (shared memory, B + 1 words).  Every thread of the block
// calls it; ends with a barrier.  scan: NT / 32 words.
template <int NT>
__device__ ChunkLine chunk_line(const ChunkParams& p, long long* before, long long* scan, int T, int KT, int unit,
                                bool report) {
  const ChunkLine line{before, p.cu_new, p.seq_lens, p.n_tokens, p.T_cap, p.B, p.Hkv, T, KT, unit};
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (p.B + NT - 1) / NT, b0 = min(p.B, tid * run), b1 = min(p.B, b0 + run);
  bool bad = false;
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    const ChunkSeq q = line.sequence(b, &bad);
    before[b] = sum;
    sum += line.cost_of(q.n, q.len);
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
  long long pre = incl - sum;
#pragma unroll
  for (int v = 0; v < NT / 32; ++v) pre += v < warp ? scan[v] : 0;
  for (int b = b0; b < b1; ++b) before[b] += pre;
  if (tid == NT - 1) before[p.B] = pre + sum;
  __syncthreads();
  return line;
}

// Place of row r of unit u in `out` and in the log-sums: its token and head.
struct ChunkRow {
  int token, head;  // of the call's rows; of the Hq heads
  __device__ ChunkRow(const ChunkParams& p, const ChunkUnit& u, int T, int r)
      : token(u.q.first + u.i * T + r / p.G), head(u.h * p.G + r % p.G) {}
  __device__ size_t out(const ChunkParams& p, int D) const { return ((size_t)token * p.Hq + head) * D; }
  __device__ size_t lse(const ChunkParams& p) const {
    return ((size_t)(head / p.G) * p.n_tokens + token) * p.G + head % p.G;
  }
};

// Whether the logits of sequence b are kept (those of its head h at chunk_logits, row after row).
__device__ __forceinline__ int light_row(const ChunkParams& p, int b, const ChunkSeq& q) {
  return p.logits_by_token ? q.first * p.G : b * CHUNK_LIGHT;
}
__device__ __forceinline__ bool chunk_light(const ChunkParams& p, int b, const ChunkSeq& q) {
  return p.logits && q.n * p.G <= CHUNK_LIGHT && light_row(p, b, q) + q.n * p.G <= p.logit_rows;
}
__device__ __forceinline__ float* chunk_logits(const ChunkParams& p, int b, int h, const ChunkSeq& q) {
  return p.logits + ((size_t)light_row(p, b, q) * p.Hkv + (size_t)h * q.n * p.G) * p.T_pad;
}

// log2 of a row's sum: infinity where it saw nothing (its weights are 0), NaN where one of its
// logits was NaN or +inf (so are its weights: a slot that it does not see is masked by index).
__device__ __forceinline__ float chunk_lse(float m, float l) { return l == 0.f ? INFINITY : m + log2f(l); }

template <typename T>
__device__ __forceinline__ void store4(T* to, float a, float b, float c, float d) {
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16(a, b), pack_bf16(c, d));
  else
    *reinterpret_cast<float4*>(to) = make_float4(a, b, c, d);
}

// V at slots that only some of a unit's tokens see: a product with a weight of 0 would bring
// what is not finite there (bits of the exponent all set) to the rows that do not see it.  So
// such elements are cleared before P V, and a row that sees one gets it here, once its result is
// stored: the element itself, since a sum with infinity or NaN does not depend on its weight.
// Slots [s0, s1) are those of the row's; to: its place, of storage type T.  Seldom called.
__device__ __forceinline__ bool not_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ void put(__nv_bfloat16* to, float x) { *to = __float2bfloat16(x); }
__device__ __forceinline__ void put(float* to, float x) { *to = x; }
template <typename T, typename O>
__device__ __noinline__ void add_not_finite(const ChunkParams& p, int b, int h, int s0, int s1, int d0, int d1, int D, O* to) {
  for (int s = s0; s < s1; ++s) {
    const long long row = paged_row(p.page_table[(size_t)b * p.max_pages + (s >> p.log2_page)], p.n_pages, p.Hkv, h, p.log2_page, s);
    if (row < 0) continue;
    for (int d = d0; d < d1; ++d) {
      const float v = as_float(static_cast<const T*>(p.v_pages)[(size_t)row * D + d]);
      if (not_finite(v)) put(to + d, as_float(to[d]) + v);
    }
  }
}
// The slots from the unit's second token's on, that its first does not see, and the end of
// those that its last one sees.
__device__ __forceinline__ int2 partly_seen(const ChunkUnit& u, int T) {
  const int a = u.q.len - u.q.n;
  return make_int2(max(0, a + u.i * T + 1), max(0, a + min((u.i + 1) * T, u.q.n)));
}

// Walks the segments of the part [y0, y1): f(unit, f0, f1, whole) for its tiles of slots
// f0 .. f1 - 1, until it says false.  The same for every role.
template <class F>
__device__ __forceinline__ void segments(const ChunkLine& line, long long y0, long long y1, F&& f) {
  ChunkUnit u;
  u.find(line, y0);
  while (true) {
    const int f0 = u.before(line, y0), f1 = u.before(line, y1);
    const bool whole = f0 == 0 && f1 == u.tiles && u.begin >= y0;
    if (f0 < f1 || whole)
      if (!f(u, f0, f1, whole)) return;
    if (u.begin + u.cost >= y1) return;
    u.next(line);
  }
}

// Record of part c: slot 0 of a unit that began before it, slot 1 of one that goes on.
__device__ __forceinline__ float* chunk_record(const ChunkParams& p, int D, int c, int slot) {
  return p.records + (size_t)(2 * c + slot) * ((size_t)p.rows * (D + 2));
}
// What the join is told of a record: the unit's first token (of the call's rows), its first
// head and its rows, and whether there is a record (1) and it is the unit's last (2).  One
// thread of each block, for both slots, before its first unit and as its segments end.
__device__ __forceinline__ void note_none(const ChunkParams& p, int c) {
  p.notes[2 * c] = p.notes[2 * c + 1] = make_int4(0, 0, 0, 0);
}
__device__ __forceinline__ void note_record(const ChunkParams& p, int c, const ChunkUnit& u, int T, int f0, int f1) {
  p.notes[2 * c + (f0 == 0)] = make_int4(u.q.first + u.i * T, u.h * p.G, min(T, u.q.n - u.i * T) * p.G,
                                         f0 > 0 && f1 == u.tiles ? 3 : 1);
}

// What is not finite among E elements of row r from d on, added up over the n parts without their
// factors (one that is too small for a number would make NaN of infinity), to the row's result.
template <int D, int E, typename T>
__device__ __noinline__ void join_not_finite(const ChunkParams& p, const int* parts, int n, int r, int d, T* to) {
  for (int e = 0; e < E; ++e) {
    float sum = 0.f;
    for (int i = 0; i < n; ++i) {
      const float x = ld_cg(chunk_record(p, D, parts[i], i == 0) + (size_t)r * D + d + e);
      if (not_finite(x)) sum += x;
    }
    if (not_finite(sum)) put(to + e, sum);
  }
}

// The units that were cut: block x takes the unit that goes on behind part x, if there is
// one, its warps the rows.  The parts of a row are added in part order.
constexpr int CJ_NT = 256;
constexpr int CJ_ROWS = 16;  // rows of a block
template <typename T, int D>
__global__ void __launch_bounds__(CJ_NT) chunk_join_kernel(const __grid_constant__ ChunkParams p) {
  __shared__ int parts[2 * CHUNK_MAX_SMS];  // that left a record of the unit, in order
  __shared__ int count;
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  paged_go();
  paged_wait();
  const int4 unit = ld_cg(p.notes + 2 * c + 1);
  const int r0 = blockIdx.y * CJ_ROWS, rows = min(unit.z, r0 + CJ_ROWS);
  if (!(unit.w & 1) || r0 >= rows) return;
  if (warp == 0) {
    int n = 1;
    if (lane == 0) parts[0] = c;
    for (int k = c + 1; k < p.parts; k += 32) {
      const int flags = k + lane < p.parts ? ld_cg(p.notes + 2 * (k + lane)).w : 0;
      const unsigned last = __ballot_sync(0xffffffffu, flags & 2);
      const unsigned mine = __ballot_sync(0xffffffffu, flags & 1) & (last ? (last & -last) * 2 - 1 : 0xffffffffu);
      if (mine >> lane & 1) parts[n + __popc(mine & ((1u << lane) - 1))] = k + lane;
      n += __popc(mine);
      if (last) break;
    }
    if (lane == 0) count = n;
  }
  __syncthreads();
  const int n = count;
  constexpr int E = D / 32, U = 4;  // U: parts that a lane has on the way
  for (int r = r0 + warp; r < rows; r += CJ_NT / 32) {
    float M = -INFINITY, L = 0.f, o[E] = {};
    for (int k0 = 0; k0 < n; k0 += U) {
      float x[U][E], m[U], l[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const bool any = k0 + i < n;
        const float* rec = chunk_record(p, D, any ? parts[k0 + i] : c, k0 + i == 0);
        m[i] = any ? ld_cg(rec + (size_t)p.rows * D + r) : -INFINITY;
        l[i] = any ? ld_cg(rec + (size_t)p.rows * (D + 1) + r) : 0.f;
        if (any) {
          if constexpr (E == 4) {
            const float4 v = ld_cg(reinterpret_cast<const float4*>(rec + (size_t)r * D) + lane);
            x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
          } else {
            x[i][0] = ld_cg(rec + (size_t)r * D + 2 * lane), x[i][1] = ld_cg(rec + (size_t)r * D + 2 * lane + 1);
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) x[i][e] = 0.f;
        }
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
    }
    const int token = unit.x + r / p.G, head = unit.y + r % p.G;
    const float inv = L > 0.f ? 1.f / L : 0.f;
    T* to = static_cast<T*>(p.out) + ((size_t)token * p.Hq + head) * D + E * lane;
    if constexpr (E == 4) store4<T>(to, o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
    else if constexpr (sizeof(T) == 2) *reinterpret_cast<uint32_t*>(to) = pack_bf16(o[0] * inv, o[1] * inv);
    else *reinterpret_cast<float2*>(to) = make_float2(o[0] * inv, o[1] * inv);
    float any = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) any += o[e];
    if (not_finite(any)) join_not_finite<D, E>(p, parts, n, r, E * lane, to);
    if (p.weight && lane == 0) p.lse[((size_t)(head / p.G) * p.n_tokens + token) * p.G + head % p.G] = chunk_lse(M, L);
  }
}

template <typename T, int D>
cudaError_t launch_chunk_join(const ChunkParams& p, cudaStream_t s) {
  if (p.parts < 2) return cudaSuccess;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.parts - 1, (p.rows + CJ_ROWS - 1) / CJ_ROWS);
  cfg.blockDim = dim3(CJ_NT);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_join_kernel<T, D>, p);
}

// A tensor of `n` dimensions (sizes and boxes from the innermost on) in the 128-byte swizzle.
inline cudaError_t tensor_map(CUtensorMap* map, const void* at, CUtensorMapDataType type, int n, const cuuint64_t* dims, const cuuint64_t* strides,
                       const cuuint32_t* box) {
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
  const cuuint32_t one[3] = {1, 1, 1};
  const CUresult r = encode(map, type, n, const_cast<void*>(at), dims, strides, box, one,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// ------------------------------------------------------------------ weights
// A unit of the weights' pass: slots [t0, t0 + SLOTS) of KV head h of sequence b, which all
// of its tokens that see them read.
struct WeightUnit {
  int b, h, t0;
  ChunkSeq q;
  __device__ int tiles(int TQ) const { return (q.n + TQ - 1) / TQ; }  // of TQ tokens
  // The first of them that sees a slot of t0 + off or behind (all of them, if there is none).
  __device__ int from(int off, int TQ) const {
    return t0 + off < q.len ? max(0, t0 + off - (q.len - q.n)) / TQ : tiles(TQ);
  }
};

// Units of one head before each sequence, in shared memory (3 (B + 1) words): of those with more
// tokens than a tile of rows holds, of the others, and of the light ones, in pieces of
// WEIGHT_PIECE slots.  Every thread of the block calls it; ends with a barrier.  scan: NT / 32
// triples of words.
constexpr int WEIGHT_PIECE = 128;
template <int NT, int SLOTS>
__device__ void weight_line(const ChunkParams& p, int* before, int3* scan, int TQ) {
  const ChunkLine line{nullptr, p.cu_new, p.seq_lens, p.n_tokens, p.T_cap, p.B, p.Hkv, 0, 0, 0};
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (p.B + NT - 1) / NT, b0 = min(p.B, tid * run), b1 = min(p.B, b0 + run);
  int* few = before + p.B + 1;
  int* light = few + p.B + 1;
  int3 sum = make_int3(0, 0, 0);
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    before[b] = sum.x;
    few[b] = sum.y;
    light[b] = sum.z;
    const ChunkSeq q = line.sequence(b, &bad);
    if (q.n > 0 && chunk_light(p, b, q)) sum.z += (q.len + WEIGHT_PIECE - 1) / WEIGHT_PIECE;
    else if (q.n > TQ) sum.x += (q.len + SLOTS - 1) / SLOTS;
    else if (q.n > 0) sum.y += (q.len + SLOTS - 1) / SLOTS;
  }
  int3 incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o),
              z = __shfl_up_sync(0xffffffffu, incl.z, o);
    if (lane >= o) {
      incl.x += x;
      incl.y += y;
      incl.z += z;
    }
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int3 pre = make_int3(incl.x - sum.x, incl.y - sum.y, incl.z - sum.z);
#pragma unroll
  for (int v = 0; v < NT / 32; ++v) {
    pre.x += v < warp ? scan[v].x : 0;
    pre.y += v < warp ? scan[v].y : 0;
    pre.z += v < warp ? scan[v].z : 0;
  }
  for (int b = b0; b < b1; ++b) {
    before[b] += pre.x;
    few[b] += pre.y;
    light[b] += pre.z;
  }
  if (tid == NT - 1) {
    before[p.B] = pre.x + sum.x;
    few[p.B] = pre.y + sum.y;
    light[p.B] = pre.z + sum.z;
  }
  __syncthreads();
}

// The sequence that holds unit x of all heads.
__device__ __forceinline__ int weight_sequence(const int* w, int B, int Hkv, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (w[mid] * Hkv <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The x-th unit; false behind the last.  A head's units fall in cost (the later the slots,
// the fewer tokens see them) and those of few tokens come last, so that blocks that take the
// next one when they are done end together (a step of two prompts and 30 single tokens, before
// light sequences kept their logits: 161 us dealt there and back, 148 so).
template <int SLOTS>
__device__ __forceinline__ bool weight_unit(const ChunkParams& p, const int* before, int x, WeightUnit& u) {
  const int first = before[p.B] * p.Hkv;
  const int* w = before;
  if (x >= first) {
    x -= first;
    w += p.B + 1;
    if (x >= w[p.B] * p.Hkv) return false;
  }
  const int lo = weight_sequence(w, p.B, p.Hkv, x);
  const ChunkLine line{nullptr, p.cu_new, p.seq_lens, p.n_tokens, p.T_cap, p.B, p.Hkv, 0, 0, 0};
  const int rem = x - w[lo] * p.Hkv;
  bool bad = false;
  u = WeightUnit{lo, rem % p.Hkv, rem / p.Hkv * SLOTS, line.sequence(lo, &bad)};
  return true;
}

// What four slots get where that is NaN for some: a log-sum of NaN goes to the slots that its row
// sees, by their index (a logit of -inf less NaN is no 0).  see: slots from the first of them on
// that the first token's rows see.  Seldom run: 16 sequences of 8000 tokens with a new one each take
// 115 us with it as without it, and 119 with the masks in the loop itself.
__device__ __forceinline__ float4 light_masked(const float* z, int T_pad, const float* lse, int rows, int G, int see) {
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int r = 0; r < rows; ++r) {
    const float4 x = ld_cg(reinterpret_cast<const float4*>(z + (size_t)r * T_pad));
    const float l = ld_cg(lse + r);
    const int n = see + r / G;
    a.x += n > 0 ? exp2f(x.x - l) : 0.f;
    a.y += n > 1 ? exp2f(x.y - l) : 0.f;
    a.z += n > 2 ? exp2f(x.z - l) : 0.f;
    a.w += n > 3 ? exp2f(x.w - l) : 0.f;
  }
  return a;
}

// The light sequences, by all warps of all blocks, a piece at a time, four slots to a lane.
template <int NT>
__device__ void weight_light(const ChunkParams& p, const int* light) {
  const ChunkLine line{nullptr, p.cu_new, p.seq_lens, p.n_tokens, p.T_cap, p.B, p.Hkv, 0, 0, 0};
  const int lane = threadIdx.x & 31, warps = gridDim.x * (NT / 32), all = light[p.B] * p.Hkv;
  for (int x = (threadIdx.x >> 5) * gridDim.x + blockIdx.x; x < all; x += warps) {
    const int b = weight_sequence(light, p.B, p.Hkv, x), rem = x - light[b] * p.Hkv, h = rem % p.Hkv;
    bool bad = false;
    const ChunkSeq q = line.sequence(b, &bad);
    const int rows = q.n * p.G, t = WEIGHT_PIECE * (rem / p.Hkv) + 4 * lane;
    if (t < q.len) {
      const int page = p.page_table[(size_t)b * p.max_pages + (t >> p.log2_page)];
      if (page < 0 || page >= p.n_pages) continue;
      const float* z = chunk_logits(p, b, h, q) + t;
      const float* lse = p.lse + ((size_t)h * p.n_tokens + q.first) * p.G;
      float4 zr[CHUNK_LIGHT];
      float l[CHUNK_LIGHT];
#pragma unroll
      for (int r = 0; r < CHUNK_LIGHT; ++r) {
        zr[r] = r < rows ? ld_cg(reinterpret_cast<const float4*>(z + (size_t)r * p.T_pad)) : make_float4(0.f, 0.f, 0.f, 0.f);
        l[r] = r < rows ? ld_cg(lse + r) : INFINITY;
      }
      float* weight = p.weight + ((size_t)b * p.Hkv + h) * p.T_cap + t;
      const float4 old = *reinterpret_cast<const float4*>(weight);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < CHUNK_LIGHT; ++r) {
        a.x += exp2f(zr[r].x - l[r]);
        a.y += exp2f(zr[r].y - l[r]);
        a.z += exp2f(zr[r].z - l[r]);
        a.w += exp2f(zr[r].w - l[r]);
      }
      const float any = (a.x + a.y) + (a.z + a.w);
      if (any != any) a = light_masked(z, p.T_pad, lse, rows, p.G, q.len - q.n + 1 - t);
      const int live = q.len - t;  // slots behind the end keep what they hold
      if (live >= 4) {
        *reinterpret_cast<float4*>(weight) = make_float4(old.x + a.x, old.y + a.y, old.z + a.z, old.w + a.w);
      } else {
        weight[0] = old.x + a.x;
        if (live > 1) weight[1] = old.y + a.y;
        if (live > 2) weight[2] = old.z + a.z;
      }
    }
  }
}

}  // namespace fasa
