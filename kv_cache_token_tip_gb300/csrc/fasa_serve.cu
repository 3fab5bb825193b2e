// Entry points of a step of new tokens over the paged cache: argument checks,
// frequencies, workspace layouts, launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>
#include <mutex>

#include "../../include/fasa.h"
#include "fasa_internal.h"
#include "fasa_serve.h"

using namespace fasa;

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t up(size_t n) { return (n + 255) & ~(size_t)255; }

// Memory that a call reads or writes.
struct Range {
  const void* p;
  size_t bytes;
};
bool apart(Range a, Range b) {
  const char *x = static_cast<const char*>(a.p), *y = static_cast<const char*>(b.p);
  return !x || !y || x + a.bytes <= y || y + b.bytes <= x;
}
bool apart(Range a, std::initializer_list<Range> all) {
  for (const Range& b : all)
    if (!apart(a, b)) return false;
  return true;
}

// The dims of the paged cache, by the check of its own entry points.
int check_dims(const fasa_paged_dims_t* d) {
  size_t bytes;
  return fasa_paged_workspace_size(d, 0, &bytes);
}

size_t pool_bytes(const fasa_paged_dims_t* d) {  // of K's or V's pages
  return (size_t)d->n_pages * d->n_kv_heads * d->page_size * d->head_dim * (d->dtype == FASA_F32 ? 4 : 2);
}
size_t stat_bytes(const fasa_paged_dims_t* d) {  // of the weights or the positions
  return (size_t)d->batch * d->n_kv_heads * d->max_pages * d->page_size * 4;
}

int log2_of(int n) {
  int k = 0;
  while ((1 << k) < n) ++k;
  return k;
}

int check_rope(const fasa_rope_t* r, int d) {
  if (!r || r->reserved) return FASA_ERR_INVALID_ARG;
  if (r->layout != FASA_ROPE_INTERLEAVED && r->layout != FASA_ROPE_HALF) return FASA_ERR_UNSUPPORTED;
  if (r->scaling < FASA_ROPE_PLAIN || r->scaling > FASA_ROPE_RAMP) return FASA_ERR_UNSUPPORTED;
  if (r->rotary_dim < 16 || r->rotary_dim > d || r->rotary_dim % 16) return FASA_ERR_INVALID_ARG;
  const auto good = [](double x) { return x > 0.0 && isfinite(x); };
  if (!good(r->rope_theta) || !good(r->magnitude) || !good((float)r->magnitude)) return FASA_ERR_INVALID_ARG;
  if (r->scaling != FASA_ROPE_PLAIN && !good(r->factor)) return FASA_ERR_INVALID_ARG;
  if (r->scaling == FASA_ROPE_WAVELENGTH || r->scaling == FASA_ROPE_RAMP)
    if (!good(r->low) || !good(r->high) || r->low >= r->high || !good(r->original)) return FASA_ERR_INVALID_ARG;
  if (r->scaling == FASA_ROPE_RAMP && r->rope_theta <= 1.0) return FASA_ERR_INVALID_ARG;
  return FASA_OK;
}

// Angle of pair i per position, radians.
double frequency(const fasa_rope_t& r, int i) {
  const double two_pi = 6.283185307179586476925286766559;
  const double t = pow(r.rope_theta, -2.0 * i / r.rotary_dim);
  const auto unit = [](double x) { return std::min(1.0, std::max(0.0, x)); };
  if (r.scaling == FASA_ROPE_LINEAR) return t / r.factor;
  if (r.scaling == FASA_ROPE_WAVELENGTH) {
    const double s = unit((r.original * t / two_pi - r.low) / (r.high - r.low));
    return t * (s + (1.0 - s) / r.factor);
  }
  if (r.scaling == FASA_ROPE_RAMP) {
    const auto index = [&](double turns) {
      return r.rotary_dim * log(r.original / (two_pi * turns)) / (2.0 * log(r.rope_theta));
    };
    const double i0 = std::max(floor(index(r.high)), 0.0), i1 = std::min(ceil(index(r.low)), r.rotary_dim - 1.0);
    const double s = unit((i - i0) / std::max(i1 - i0, 0.001));
    return t * (1.0 - s + s / r.factor);
  }
  return t;
}

// The pairs' angles in 2^-64 turns (those of the last call are kept: 64 powers take
// longer than a launch).
void turns_of(const fasa_rope_t& r, unsigned long long (&turns)[64]) {
  static std::mutex mu;
  static fasa_rope_t last;
  static unsigned long long kept[64];
  static bool any = false;
  std::lock_guard<std::mutex> lk(mu);
  if (!any || memcmp(&last, &r, sizeof(r))) {
    const long double two64_over_2pi = 18446744073709551616.0L / 6.28318530717958647692528676655900577L;
    memset(kept, 0, sizeof(kept));
    for (int i = 0; i < r.rotary_dim / 2; ++i) {
      const long double x = (long double)frequency(r, i) * two64_over_2pi;  // (whole turns fall away)
      kept[i] = (unsigned long long)fmodl(x, 18446744073709551616.0L);
    }
    last = r;
    any = true;
  }
  memcpy(turns, kept, sizeof(kept));
}

// Rows of a record, and the most parts that the work can come to.
void chunk_plan(const fasa_paged_dims_t* d, int n_tokens, int sms, int* rows, int* parts) {
  const int G = d->n_q_heads / d->n_kv_heads;
  const ChunkShape s = chunk_shape(d->dtype == FASA_BF16, G);
  const int T = s.tokens;
  // (whole 16-byte words to a record)
  *rows = ((int)std::min<long long>((long long)T * G, (long long)n_tokens * G) + 3) / 4 * 4;
  // a part without a tile has nothing to do: no more parts than units of the longest cache have tiles
  const long long units = ((long long)n_tokens / T + std::min(d->batch, n_tokens)) * d->n_kv_heads;
  const long long tiles = ((long long)d->max_pages * d->page_size + T + s.tile - 1) / s.tile + 1;
  *parts = (int)std::min<long long>(std::min(sms, CHUNK_MAX_SMS), units * tiles);
}

size_t notes_bytes(int parts) { return 256 + up((size_t)parts * 2 * sizeof(int4)); }  // and the queue
int padded_slots(const fasa_paged_dims_t* d) { return (d->max_pages * d->page_size + 127) / 128 * 128; }
// Rows of the light sequences' logits, were they all kept, and whether they lie by token.
long long light_rows(const fasa_paged_dims_t* d, int n_tokens, bool* by_token) {
  const long long tokens = (long long)n_tokens * (d->n_q_heads / d->n_kv_heads), all = (long long)d->batch * CHUNK_LIGHT;
  *by_token = tokens < all;
  return std::min(tokens, all);
}
long long logit_row_bytes(const fasa_paged_dims_t* d) { return (long long)d->n_kv_heads * padded_slots(d) * 4; }
// Logits of the light sequences, where there is a second pass that reads them.
size_t logits_bytes(const fasa_paged_dims_t* d, int n_tokens) {
  bool by_token;
  return up((size_t)std::min(light_rows(d, n_tokens, &by_token) * logit_row_bytes(d), CHUNK_LOGITS));
}
size_t records_bytes(int rows, int parts, int D) { return up((size_t)parts * 2 * rows * (D + 2) * 4); }

}  // namespace

extern "C" {

int fasa_paged_assign(const int32_t* have_lens, const int32_t* want_lens, const int32_t* pos, int32_t* page_table,
                      int32_t* free_pages, const int32_t* free_count, int32_t* lens_out, int32_t* free_count_out,
                      int32_t* cu_new, int32_t* token_map, int32_t max_tokens, const fasa_paged_dims_t* dims,
                      fasa_stream_t stream) {
  int st = check_dims(dims);
  if (st) return st;
  if (!have_lens || !want_lens || !page_table || !free_pages || !free_count || !lens_out || !free_count_out || !cu_new)
    return FASA_ERR_INVALID_ARG;
  if (max_tokens < 0 || (max_tokens > 0 && !token_map) || !aligned(token_map, 16)) return FASA_ERR_INVALID_ARG;
  if (max_tokens > ASSIGN_MAX_TOKENS) return FASA_ERR_UNSUPPORTED;
  for (const void* x : {(const void*)have_lens, (const void*)want_lens, (const void*)pos, (const void*)page_table,
                        (const void*)free_pages, (const void*)free_count, (const void*)lens_out,
                        (const void*)free_count_out, (const void*)cu_new})
    if (!aligned(x, 4)) return FASA_ERR_INVALID_ARG;
  const size_t lens = (size_t)dims->batch * 4;
  const Range have{have_lens, lens}, want{want_lens, lens}, at{pos, lens}, count{free_count, 4},
      table{page_table, lens * dims->max_pages}, list{free_pages, (size_t)dims->n_pages * 4}, out{lens_out, lens},
      left{free_count_out, 4}, cu{cu_new, lens + 4}, map{token_map, (size_t)max_tokens * 16};
  // every block reads the first four; the lengths and the count go out when all have
  if (!apart(table, {have, want, at, count, list, out, left, cu, map}) ||
      !apart(list, {have, want, at, count, out, left, cu, map}) || !apart(cu, {have, want, at, count, out, left, map}) ||
      !apart(map, {have, want, at, count, out, left}) || !apart(out, {at, count, left}) || !apart(left, {have, want, at}))
    return FASA_ERR_INVALID_ARG;
  if ((lens_out != have_lens && !apart(out, have)) || (lens_out != want_lens && !apart(out, want)))
    return FASA_ERR_INVALID_ARG;
  int sms = 0, *status = nullptr;
  st = device_facts(&sms, &status);
  if (st) return st;
  AssignParams p;
  p.B = dims->batch;
  p.max_pages = dims->max_pages;
  p.log2_page = log2_of(dims->page_size);
  p.n_pages = dims->n_pages;
  p.T_cap = dims->max_pages * dims->page_size;
  p.max_tokens = max_tokens;
  p.have = have_lens;
  p.want = want_lens;
  p.pos = pos;
  p.page_table = page_table;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.lens_out = lens_out;
  p.free_count_out = free_count_out;
  p.cu_new = cu_new;
  p.token_map = reinterpret_cast<int4*>(token_map);
  p.status = status;
  const cudaError_t e = launch_paged_assign(p, sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FASA_OK : report_cuda(e);
}

int fasa_paged_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, const int32_t* token_map, int32_t n_tokens, void* q_out, void* k_pages,
                           void* v_pages, float* weight, int32_t* token_pos, const fasa_rope_t* rope,
                           const fasa_paged_dims_t* dims, fasa_stream_t stream) {
  int st = check_dims(dims);
  if (st) return st;
  st = check_rope(rope, dims->head_dim);
  if (st) return st;
  if (n_tokens < 0) return FASA_ERR_INVALID_ARG;
  if (n_tokens > ASSIGN_MAX_TOKENS) return FASA_ERR_UNSUPPORTED;
  if (n_tokens == 0) return FASA_OK;  // (tensors without rows have no addresses)
  if (!q != !q_out || !k != !v || !k != !k_pages || !k != !v_pages || (!k && (weight || token_pos)))
    return FASA_ERR_INVALID_ARG;
  if (!q && !k) return FASA_OK;
  if (!token_map) return FASA_ERR_INVALID_ARG;
  for (const void* x : {q, k, v, (const void*)token_map, (const void*)q_out, (const void*)k_pages, (const void*)v_pages,
                        (const void*)weight, (const void*)token_pos})
    if (!aligned(x, 16)) return FASA_ERR_INVALID_ARG;
  const int es = dims->dtype == FASA_F32 ? 4 : 2;
  const int64_t heads[3] = {dims->n_q_heads, dims->n_kv_heads, dims->n_kv_heads}, strides[3] = {q_stride, k_stride, v_stride};
  const void* from[3] = {q, k, v};
  Range in[3];
  for (int i = 0; i < 3; ++i) {
    in[i] = {from[i], 0};
    if (!from[i]) continue;
    const int64_t row = heads[i] * dims->head_dim;
    if (strides[i] < row || strides[i] > ((int64_t)1 << 32) || strides[i] * es % 16) return FASA_ERR_INVALID_ARG;
    in[i].bytes = (size_t)((n_tokens - 1) * strides[i] + row) * es;
  }
  const int64_t row = heads[0] * dims->head_dim;
  const Range out{q_out, q ? (size_t)n_tokens * row * es : 0};
  if (q && !(q_out == q && q_stride == row) && !apart(out, in[0])) return FASA_ERR_INVALID_ARG;
  // a token's rows are read and written by its own warps, in no order among tokens
  const Range map{token_map, (size_t)n_tokens * 16}, keys{k_pages, pool_bytes(dims)}, values{v_pages, pool_bytes(dims)},
      given{weight, stat_bytes(dims)}, at{token_pos, stat_bytes(dims)};
  if (!apart(out, {in[1], in[2], map, keys, values, given, at}) || !apart(keys, {in[0], in[1], in[2], map, values, given, at}) ||
      !apart(values, {in[0], in[1], in[2], map, given, at}) || !apart(given, {in[0], in[1], in[2], map, at}) ||
      !apart(at, {in[0], in[1], in[2], map}))
    return FASA_ERR_INVALID_ARG;
  int sms = 0, *status = nullptr;
  st = device_facts(&sms, &status);
  if (st) return st;
  RopeAppendParams p;
  turns_of(*rope, p.turns);
  p.magnitude = (float)rope->magnitude;
  p.rotary_dim = rope->rotary_dim;
  p.n_tokens = n_tokens;
  p.B = dims->batch;
  p.Hq = dims->n_q_heads;
  p.Hkv = dims->n_kv_heads;
  p.log2_page = log2_of(dims->page_size);
  p.n_pages = dims->n_pages;
  p.T_cap = dims->max_pages * dims->page_size;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.token_map = reinterpret_cast<const int4*>(token_map);
  p.q_out = q_out;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.weight = weight;
  p.token_pos = token_pos;
  p.status = status;
  const cudaError_t e = launch_rope_append(p, dims->head_dim, dims->dtype == FASA_BF16, rope->layout == FASA_ROPE_HALF,
                                           sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FASA_OK : report_cuda(e);
}

int fasa_paged_chunk_workspace_size(const fasa_paged_dims_t* dims, int32_t n_tokens, int32_t with_weight,
                                    size_t* bytes) {
  if (!bytes) return FASA_ERR_INVALID_ARG;
  *bytes = 0;
  const int st = check_dims(dims);
  if (st) return st;
  if (n_tokens < 0) return FASA_ERR_INVALID_ARG;
  if (n_tokens > CHUNK_MAX_TOKENS) return FASA_ERR_UNSUPPORTED;
  if (n_tokens == 0) return FASA_OK;
  int rows, parts;  // (of any device)
  chunk_plan(dims, n_tokens, CHUNK_MAX_SMS, &rows, &parts);
  *bytes = notes_bytes(parts) + records_bytes(rows, parts, dims->head_dim);
  if (with_weight) *bytes += logits_bytes(dims, n_tokens) + up((size_t)n_tokens * dims->n_q_heads * 4);
  return FASA_OK;
}

int fasa_paged_chunk_attention(const void* q, int32_t n_tokens, const int32_t* cu_new, const void* k_pages,
                               const void* v_pages, const int32_t* page_table, const int32_t* seq_lens, void* out,
                               float* weight, void* workspace, size_t workspace_bytes,
                               const fasa_paged_dims_t* dims, fasa_stream_t stream) {
  size_t need = 0;
  int st = fasa_paged_chunk_workspace_size(dims, n_tokens, weight != nullptr, &need);
  if (st) return st;
  if (!cu_new && n_tokens != dims->batch) return FASA_ERR_INVALID_ARG;
  if (!k_pages || !v_pages || !page_table || !seq_lens) return FASA_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!q || !out)) return FASA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) || !aligned(weight, 16))
    return FASA_ERR_INVALID_ARG;
  if (n_tokens == 0) return FASA_OK;
  for (const void* x : {(const void*)cu_new, (const void*)page_table, (const void*)seq_lens})
    if (!aligned(x, 4)) return FASA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return FASA_ERR_WORKSPACE;
  // Rows, lengths and pages are read again and again, by roles that have to agree on them, while
  // results, weights and workspace are written
  const size_t es = dims->dtype == FASA_F32 ? 4 : 2, io = (size_t)n_tokens * dims->n_q_heads * dims->head_dim * es;
  const Range query{q, io}, cu{cu_new, (size_t)dims->batch * 4 + 4}, keys{k_pages, pool_bytes(dims)}, values{v_pages, pool_bytes(dims)},
      table{page_table, (size_t)dims->batch * dims->max_pages * 4}, lens{seq_lens, (size_t)dims->batch * 4}, result{out, io},
      given{weight, stat_bytes(dims)}, room{workspace, need};
  if (!apart(result, {query, cu, keys, values, table, lens, given, room}) ||
      !apart(given, {query, cu, keys, values, table, lens, room}) || !apart(room, {query, cu, keys, values, table, lens}))
    return FASA_ERR_INVALID_ARG;
  int sms = 0, *status = nullptr;
  st = device_facts(&sms, &status);
  if (st) return st;
  ChunkParams p;
  p.B = dims->batch;
  p.Hq = dims->n_q_heads;
  p.Hkv = dims->n_kv_heads;
  p.G = p.Hq / p.Hkv;
  p.log2_page = log2_of(dims->page_size);
  p.n_pages = dims->n_pages;
  p.max_pages = dims->max_pages;
  p.T_cap = dims->max_pages * dims->page_size;
  p.n_tokens = n_tokens;
  p.q = q;
  p.cu_new = cu_new;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.out = out;
  p.weight = weight;
  p.scale = (float)(1.4426950408889634 / sqrt((double)dims->head_dim));
  chunk_plan(dims, n_tokens, sms, &p.rows, &p.parts);
  p.sms = sms;
  char* ws = static_cast<char*>(workspace);
  p.queue = reinterpret_cast<int*>(ws);
  p.notes = reinterpret_cast<int4*>(ws + 256);
  ws += notes_bytes(p.parts);
  p.records = reinterpret_cast<float*>(ws);
  ws += records_bytes(p.rows, p.parts, dims->head_dim);
  p.T_pad = padded_slots(dims);
  p.logits = weight ? reinterpret_cast<float*>(ws) : nullptr;
  p.logit_rows = (int)std::min(light_rows(dims, n_tokens, &p.logits_by_token), CHUNK_LOGITS / logit_row_bytes(dims));
  p.lse = reinterpret_cast<float*>(ws + (weight ? logits_bytes(dims, n_tokens) : 0));
  p.status = status;
  p.wait_ns = wait_limit_ns();
  p.drop_tile = dropped_copy();
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dims->dtype == FASA_BF16 ? launch_chunk_bf16(p, dims->head_dim, s) : launch_chunk_f32(p, dims->head_dim, s);
  return e == cudaSuccess ? FASA_OK : report_cuda(e);
}

}  // extern "C"
