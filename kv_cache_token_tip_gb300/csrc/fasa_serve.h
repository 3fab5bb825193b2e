// Internal definitions of a step of new tokens over the paged cache: launch
// parameters, workspace layouts and launchers (fasa_serve.cu checks arguments and
// calls them).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fasa_chunk_index.h"
#include "fasa_paged.h"

namespace fasa {

constexpr int ASSIGN_MAX_TOKENS = 1 << 24;
constexpr int CHUNK_MAX_TOKENS = 1 << 20;

struct AssignParams {
  int B, max_pages, log2_page, n_pages, T_cap, max_tokens;
  const int* have;
  const int* want;
  const int* pos;  // null: a token's slot
  int* page_table;
  int* free_pages;
  const int* free_count;
  int* lens_out;
  int* free_count_out;
  int* cu_new;
  int4* token_map;
  int* status;
};

struct RopeAppendParams {
  unsigned long long turns[64];  // of pair i per position, 2^64 to a turn
  float magnitude;
  int rotary_dim, n_tokens;
  int B, Hq, Hkv, log2_page, n_pages, T_cap;
  const void* q;  // null: no queries
  const void* k;  // null: no keys and values
  const void* v;
  long long q_stride, k_stride, v_stride;
  const int4* token_map;
  void* q_out;
  void* k_pages;
  void* v_pages;
  float* weight;
  int* token_pos;
  int* status;
};

// The attention of chunks.  Workspace: the parts' records (two per part: a unit that
// began in an earlier part, a unit that goes on in a later one) with a note to each and the
// queue of the weights' pass, and with weights the light sequences' logits and the rows'
// log-sums.
struct ChunkParams {
  int B, Hq, Hkv, G, log2_page, n_pages, max_pages, T_cap, n_tokens;
  const void* q;
  const int* cu_new;  // null: a token a sequence
  const void* k_pages;
  const void* v_pages;
  const int* page_table;
  const int* seq_lens;
  void* out;
  float* weight;   // null: no weights kept
  float scale;     // log2(e) / sqrt(d): logits are kept in powers of two
  float* records;  // [parts][2][rows * (d + 2)]: o [rows][d], m [rows], l [rows]
  int4* notes;     // [parts][2]: whose the records are
  float* logits;   // [logit_rows][Hkv] of T_pad, those of sequences of few rows; null: not kept
  int logit_rows;  // that there is room for
  bool logits_by_token;  // a token has the rows of its own place; else a sequence has CHUNK_LIGHT
  int T_pad;       // T_cap in whole tiles of slots
  int* queue;      // the next unit of the weights' pass (the first kernel sets it to 0)
  float* lse;      // [Hkv][n_tokens * G]
  int rows;        // of a record
  int parts;       // most parts of this launch
  int sms;
  int* status;
  unsigned long long wait_ns;
  int drop_tile;  // test hook: this tile of every part is never copied (-1: none)
};

// A sequence is light with this many rows (new tokens times the heads of a group) or fewer: its
// logits are kept for the weights, 16 bytes a slot for 4 rows instead of K's 256 again, as far as
// CHUNK_LOGITS bytes go: the first sequences' then, so that a larger batch or table never needs a
// smaller workspace.  Room is for the tokens' rows, or for CHUNK_LIGHT a sequence where that is
// less (a step with prompts).  With 4, 8 and 16 rows, groups of 4 heads, bf16: 16 sequences of 8000
// tokens with 1 new one 111, 112 and 115 us, with 2 201, 118 and 119, with 4 205, 204 and 131; fp32,
// 1076, 1076 and 1080, 1480, 1311 and 1313, 1483, 1483 and 1328.
constexpr int CHUNK_LIGHT = 16;
constexpr long long CHUNK_LOGITS = 480ll << 20;

cudaError_t launch_paged_assign(const AssignParams& p, int sms, cudaStream_t s);
cudaError_t launch_rope_append(const RopeAppendParams& p, int head_dim, bool bf16, bool half, int sms, cudaStream_t s);
cudaError_t launch_chunk_f32(const ChunkParams& p, int head_dim, cudaStream_t s);
cudaError_t launch_chunk_bf16(const ChunkParams& p, int head_dim, cudaStream_t s);

}  // namespace fasa
