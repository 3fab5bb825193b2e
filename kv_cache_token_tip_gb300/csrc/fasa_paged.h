// Internal definitions of the paged cache: launch parameters, workspace
// layouts and launchers (fasa_paged.cu checks arguments and calls them).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

#include "fasa_paged_index.h"

namespace fasa {

// From fasa_api.cu: theta_i / (2 pi) as 64-bit fixed-point turns; the current
// device's SM count and status word (a FASA_* code); keeps a CUDA error for
// fasa_last_cuda_error and returns FASA_ERR_CUDA.
void rope_turns_table(double rope_theta, int head_dim, unsigned long long (&turns)[64]);
int device_facts(int* sms, int** status);
int report_cuda(cudaError_t e);
unsigned long long wait_limit_ns();  // bound of every device wait
int dropped_copy();                  // test hook: the copy that is left unissued (-1: none)

struct PagedCommon {
  int B, Hq, Hkv, G, log2_page, n_pages, max_pages, T_cap;
  const int* page_table;
  const int* seq_lens;
  const int* pos;
  int* status;
};

struct PagedAppendParams : PagedCommon {
  unsigned long long rope_turns[64];
  const void* k_new;
  const void* v_new;
  int n_tokens;
  const int* cu_new;  // null: token b belongs to sequence b
  void* k_pages;
  void* v_pages;
  float* weight;   // null: not kept
  int* token_pos;  // null: not kept
};

// Attention workspace: the parts' records (two per part: a unit that began in
// an earlier part, a unit that goes on in a later one), and with weights the
// units' log-sums and every token's logits.
struct PagedAttendParams : PagedCommon {
  unsigned long long rope_turns[64];
  const void* q;
  const void* k_pages;
  const void* v_pages;
  float* out;
  float* weight;  // null: no weights kept
  float scale;    // log2(e) / sqrt(d): logits are kept in powers of two
  float* records; // [parts][2][G * (d + 2)]: o [G][d], then m [G], l [G]
  float* lse;     // [units][G] of the units one part holds whole
  float* logits;  // [units][T_cap / 16][G][16]
  int parts;      // most parts of this launch
  unsigned long long wait_ns;  // bound of every device wait
  int drop_group;              // test hook: this group of part 0 is never copied (-1: none)
};

// A token that an eviction moves: row in the pool and slot, the hole's and its own.
struct alignas(16) PagedMove {
  int2 hole, mover;
};

struct PagedEvictParams : PagedCommon {
  const float* weight;
  const int* token_pos;
  void* k_pages;
  void* v_pages;
  float* weight_out;
  int* token_pos_out;
  int* new_lens;
  int keep, sinks, recent;
  PagedMove* moves;  // [units][move_cap]
  int move_cap;
  int row_bytes;   // of a K or V row
};

// (whole 16-byte words, so that the next record begins on a boundary)
FASA_HD int paged_record_floats(int G, int D) { return (G * (D + 2) + 3) / 4 * 4; }
// A kernel of the paged cache begins under the tail of the kernel before it in its
// stream (paged_behind: the launch), waits for all that came before its first
// access to memory (paged_wait: every thread of every block) and lets the next
// kernel begin as early (paged_go).  A kernel may read ahead of its wait only what
// is older than the kernel before it, and past L1 (ld_cg): so where that one goes on
// before it waits, nothing.  The launch of one such kernel behind another then costs
// little.
template <class... P, class... A>
cudaError_t paged_behind(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, unsigned cluster,
                         cudaStream_t s, A&&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}
#ifdef __CUDACC__
__device__ __forceinline__ void paged_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void paged_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Loads past L1 that stay behind a wait or a barrier (the __ldg and __ldcg functions
// may be taken for loads of what never changes, and moved ahead of it).
__device__ __forceinline__ int ld_cg(const int* p) {
  int v;
  asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float ld_cg(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ int4 ld_cg(const int4* p) {
  int4 v;
  asm volatile("ld.global.cg.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ float4 ld_cg(const float4* p) {
  float4 v;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld_cg(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
#endif

size_t paged_attend_workspace(int units, int G, int D, int T_cap, bool weights);
void paged_attend_layout(PagedAttendParams& p, int units, int D, void* ws);

cudaError_t launch_paged_append(const PagedAppendParams& p, int head_dim, bool bf16, int sms, cudaStream_t s);
cudaError_t launch_paged_attend(const PagedAttendParams& p, int head_dim, bool bf16, int sms, cudaStream_t s);
cudaError_t launch_paged_evict(const PagedEvictParams& p, int sms, cudaStream_t s);

}  // namespace fasa
