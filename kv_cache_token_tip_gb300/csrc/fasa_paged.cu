// Entry points of the paged cache: argument checks, workspace layouts, launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "../../include/fasa.h"
#include "fasa_internal.h"
#include "fasa_paged.h"

using namespace fasa;

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_paged_dims(const fasa_paged_dims_t* d) {
  if (!d) return FASA_ERR_INVALID_ARG;
  if (d->batch < 1 || d->n_q_heads < 1 || d->n_kv_heads < 1) return FASA_ERR_INVALID_ARG;
  if (d->n_q_heads % d->n_kv_heads) return FASA_ERR_INVALID_ARG;
  if (d->head_dim < 2 || (d->head_dim & 1)) return FASA_ERR_INVALID_ARG;
  if (d->page_size < 1 || d->n_pages < 1 || d->max_pages < 1) return FASA_ERR_INVALID_ARG;
  if (!(d->rope_theta > 0.0) || !isfinite(d->rope_theta)) return FASA_ERR_INVALID_ARG;
  if (d->dtype != FASA_F32 && d->dtype != FASA_BF16) return FASA_ERR_UNSUPPORTED;
  if (d->head_dim != 64 && d->head_dim != 128) return FASA_ERR_UNSUPPORTED;
  if (d->n_q_heads / d->n_kv_heads > G_MAX) return FASA_ERR_UNSUPPORTED;
  if (d->page_size < 16 || d->page_size > 256 || (d->page_size & (d->page_size - 1))) return FASA_ERR_UNSUPPORTED;
  if (d->batch > PAGED_MAX_BATCH || (long long)d->batch * d->n_kv_heads > 65535) return FASA_ERR_UNSUPPORTED;
  if ((long long)d->max_pages * d->page_size > PAGED_MAX_SLOTS) return FASA_ERR_UNSUPPORTED;
  if ((long long)d->n_pages * d->n_kv_heads * d->page_size > 0x7fffffffll) return FASA_ERR_UNSUPPORTED;
  return FASA_OK;
}

void fill(PagedCommon& p, const fasa_paged_dims_t* d, const int32_t* page_table, const int32_t* seq_lens,
          const int32_t* pos, int* status) {
  p.B = d->batch;
  p.Hq = d->n_q_heads;
  p.Hkv = d->n_kv_heads;
  p.G = d->n_q_heads / d->n_kv_heads;
  p.log2_page = 0;
  while ((1 << p.log2_page) < d->page_size) ++p.log2_page;
  p.n_pages = d->n_pages;
  p.max_pages = d->max_pages;
  p.T_cap = d->max_pages * d->page_size;
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.pos = pos;
  p.status = status;
}

size_t up(size_t n) { return (n + 255) & ~(size_t)255; }

// Moves a unit may need: no more than slots below `keep`, nor than slots behind it.
int most_moves(const fasa_paged_dims_t* d, int keep) {
  return std::max(0, std::min(keep, d->max_pages * d->page_size - keep));
}

bool apart(const void* a, const void* b, size_t a_bytes, size_t b_bytes) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return x + a_bytes <= y || y + b_bytes <= x;
}
bool apart(const void* a, const void* b, size_t bytes) { return apart(a, b, bytes, bytes); }

}  // namespace

namespace fasa {

size_t paged_attend_workspace(int units, int G, int D, int T_cap, bool weights) {
  size_t n = up((size_t)PAGED_MAX_PARTS * 2 * paged_record_floats(G, D) * 4);
  if (weights) n += up((size_t)units * G * 4) + up((size_t)units * G * T_cap * 4);
  return n;
}

void paged_attend_layout(PagedAttendParams& p, int units, int D, void* ws) {
  char* w = static_cast<char*>(ws);
  p.records = reinterpret_cast<float*>(w);
  w += up((size_t)PAGED_MAX_PARTS * 2 * paged_record_floats(p.G, D) * 4);
  p.lse = reinterpret_cast<float*>(w);
  w += up((size_t)units * p.G * 4);
  p.logits = reinterpret_cast<float*>(w);
}

}  // namespace fasa

extern "C" {

int fasa_paged_append(const void* k_new, const void* v_new, int32_t n_tokens, const int32_t* cu_new,
                      const int32_t* pos, const int32_t* page_table, const int32_t* seq_lens, void* k_pages,
                      void* v_pages, float* weight, int32_t* token_pos, const fasa_paged_dims_t* dims,
                      fasa_stream_t stream) {
  int st = check_paged_dims(dims);
  if (st) return st;
  if (n_tokens < 0 || (!cu_new && n_tokens != dims->batch)) return FASA_ERR_INVALID_ARG;
  if (!pos || !page_table || !seq_lens || !k_pages || !v_pages) return FASA_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!k_new || !v_new)) return FASA_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
      !aligned(weight, 16) || !aligned(token_pos, 16))
    return FASA_ERR_INVALID_ARG;
  if (n_tokens == 0) return FASA_OK;
  int sms = 0, *status = nullptr;
  st = device_facts(&sms, &status);
  if (st) return st;
  PagedAppendParams p;
  fill(p, dims, page_table, seq_lens, pos, status);
  rope_turns_table(dims->rope_theta, dims->head_dim, p.rope_turns);
  p.k_new = k_new;
  p.v_new = v_new;
  p.n_tokens = n_tokens;
  p.cu_new = cu_new;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.weight = weight;
  p.token_pos = token_pos;
  const cudaError_t e =
      launch_paged_append(p, dims->head_dim, dims->dtype == FASA_BF16, sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FASA_OK : report_cuda(e);
}

int fasa_paged_workspace_size(const fasa_paged_dims_t* dims, int32_t with_weight, size_t* bytes) {
  if (!bytes) return FASA_ERR_INVALID_ARG;
  *bytes = 0;
  const int st = check_paged_dims(dims);
  if (st) return st;
  *bytes = paged_attend_workspace(dims->batch * dims->n_kv_heads, dims->n_q_heads / dims->n_kv_heads,
                                  dims->head_dim, dims->max_pages * dims->page_size, with_weight != 0);
  return FASA_OK;
}

int fasa_paged_attention(const void* q, const int32_t* pos, const void* k_pages, const void* v_pages,
                         const int32_t* page_table, const int32_t* seq_lens, float* out, float* weight,
                         void* workspace, size_t workspace_bytes, const fasa_paged_dims_t* dims,
                         fasa_stream_t stream) {
  size_t need = 0;
  int st = fasa_paged_workspace_size(dims, weight != nullptr, &need);
  if (st) return st;
  if (!q || !pos || !k_pages || !v_pages || !page_table || !seq_lens || !out) return FASA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) || !aligned(weight, 16))
    return FASA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return FASA_ERR_WORKSPACE;
  int sms = 0, *status = nullptr;
  st = device_facts(&sms, &status);
  if (st) return st;
  PagedAttendParams p;
  fill(p, dims, page_table, seq_lens, pos, status);
  rope_turns_table(dims->rope_theta, dims->head_dim, p.rope_turns);
  p.q = q;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.out = out;
  p.weight = weight;
  p.wait_ns = wait_limit_ns();
  p.drop_group = dropped_copy();
  p.scale = (float)(1.4426950408889634 / sqrt((double)dims->head_dim));
  paged_attend_layout(p, dims->batch * dims->n_kv_heads, dims->head_dim, workspace);
  const cudaError_t e =
      launch_paged_attend(p, dims->head_dim, dims->dtype == FASA_BF16, sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FASA_OK : report_cuda(e);
}

int fasa_paged_evict_workspace_size(const fasa_paged_dims_t* dims, int32_t keep, size_t* bytes) {
  if (!bytes) return FASA_ERR_INVALID_ARG;
  *bytes = 0;
  const int st = check_paged_dims(dims);
  if (st) return st;
  if (keep < 1) return FASA_ERR_INVALID_ARG;
  *bytes = up((size_t)dims->batch * dims->n_kv_heads * most_moves(dims, keep) * sizeof(PagedMove));
  return FASA_OK;
}

int fasa_paged_evict(const float* weight, const int32_t* token_pos, const int32_t* pos, const int32_t* page_table,
                     const int32_t* seq_lens, int32_t keep, int32_t sinks, int32_t recent, void* k_pages,
                     void* v_pages, float* weight_out, int32_t* token_pos_out, int32_t* new_lens, void* workspace,
                     size_t workspace_bytes, const fasa_paged_dims_t* dims, fasa_stream_t stream) {
  size_t need = 0;
  int st = fasa_paged_evict_workspace_size(dims, keep, &need);
  if (st) return st;
  if (!weight || !token_pos || !pos || !page_table || !seq_lens || !k_pages || !v_pages || !weight_out ||
      !token_pos_out || !new_lens)
    return FASA_ERR_INVALID_ARG;
  if (sinks < 0 || recent < 0 || (long long)sinks + recent > keep) return FASA_ERR_INVALID_ARG;
  // new_lens is written while other heads' blocks still read these
  const size_t lens = (size_t)dims->batch * 4;
  if (!apart(new_lens, seq_lens, lens, lens) || !apart(new_lens, pos, lens, lens) ||
      !apart(new_lens, page_table, lens, lens * dims->max_pages))
    return FASA_ERR_INVALID_ARG;
  if (!aligned(weight, 16) || !aligned(token_pos, 16) || !aligned(weight_out, 16) || !aligned(token_pos_out, 16) ||
      !aligned(k_pages, 16) || !aligned(v_pages, 16))
    return FASA_ERR_INVALID_ARG;
  // the statistics in place, both of them, or apart
  const size_t stat = (size_t)dims->batch * dims->n_kv_heads * dims->max_pages * dims->page_size * 4;
  if ((weight_out == weight) != (token_pos_out == token_pos)) return FASA_ERR_INVALID_ARG;
  if (weight_out != weight &&
      (!apart(weight_out, weight, stat) || !apart(weight_out, token_pos, stat) || !apart(token_pos_out, weight, stat) ||
       !apart(token_pos_out, token_pos, stat)))
    return FASA_ERR_INVALID_ARG;
  if (!apart(weight_out, token_pos_out, stat)) return FASA_ERR_INVALID_ARG;
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return FASA_ERR_WORKSPACE;
  int sms = 0, *status = nullptr;
  st = device_facts(&sms, &status);
  if (st) return st;
  PagedEvictParams p;
  fill(p, dims, page_table, seq_lens, pos, status);
  p.weight = weight;
  p.token_pos = token_pos;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.weight_out = weight_out;
  p.token_pos_out = token_pos_out;
  p.new_lens = new_lens;
  p.keep = keep;
  p.sinks = sinks;
  p.recent = recent;
  p.moves = static_cast<PagedMove*>(workspace);
  p.move_cap = most_moves(dims, keep);
  p.row_bytes = dims->head_dim * (dims->dtype == FASA_F32 ? 4 : 2);
  const cudaError_t e = launch_paged_evict(p, sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FASA_OK : report_cuda(e);
}

}  // extern "C"
