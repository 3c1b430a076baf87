// Internal launch interface of the batched paged step's kernels (page plan,
// rotary rows and append, chunk attention, draft verification).
#pragma once
#include "kernels.h"

namespace dvlm {

// Verification of drafted tokens by rejection sampling (csrc/spec_sample.cu).
struct SpecSampleArgs {
  const void* target_p;       // [b][K + 1][V] fp32 or bf16
  const void* draft_p;        // [b][K][V], or NULL: all of a draft's probability on its token
  const int32_t* draft_ids;   // [b][K]
  const int32_t* n_draft;     // [b] drafts of each sequence (NULL: K)
  const float* u_accept;      // [b][K]
  const float* u_sample;      // [b]
  int b, K, V;
  int32_t* accept_len;        // [b]
  int32_t* out_ids;           // [b][K + 1]
  const int32_t* cache_len;   // [b] (NULL with cache_len_out)
  int32_t* cache_len_out;
  const int32_t* cu_rows;     // [b + 1] row offsets of the step that ran, or NULL: every sequence ran
  int* status;
};
cudaError_t launch_spec_sample(const SpecSampleArgs& a, bool is_bf16, cudaStream_t s);

// Page plan of one ragged step (csrc/page_plan.cu).
constexpr int kPlanMaxBatch = 4096;
struct PagePlanArgs {
  const int32_t* cache_len;   // [n_batch] cached slots
  const int32_t* new_len;     // [n_batch] rows of this step; -1: finished
  int32_t* block_table;       // [n_batch][max_pages]
  int32_t* free_pages;        // [n_pages] stack, top at *free_count - 1
  const int32_t* free_count;
  int n_batch, max_pages, n_pages, max_rows;
  int32_t* kv_len;            // [n_batch]
  int32_t* cu_rows;           // [n_batch + 1]
  int32_t* slot_map;          // [max_rows]
  int32_t* free_count_out;
  int32_t* held_len;          // [n_batch] slots whose pages a request holds (in/out), or NULL: cache_len
  int in_place;               // some output is an input array
  int* status;
};
cudaError_t launch_page_plan(const PagePlanArgs& a, cudaStream_t s);

// Rotary positions with several axes (csrc/mrope.cu).
constexpr int kMropeMaxAxes = 4;
struct MropeAxes {
  const int32_t* pos;         // [n][n_rows]
  int n;
  int section[kMropeMaxAxes]; // frequencies of each axis, rot / 2 together
  int interleaved;
  int rot;                    // turned elements of a head (the first rot)
  double log2_base;
};
cudaError_t launch_mrope_rows(const void* x, void* out, long long x_ld, long long out_ld, int n_rows, int n_heads,
                              int D, bool is_bf16, const MropeAxes& ax, cudaStream_t s);
struct MropeAppendArgs {
  const bf16* qkv;            // [n_rows][qkv_ld]: Hq + 2 Hkv heads
  long long qkv_ld;
  bf16* q_out;                // [n_rows][Hq][D]
  bf16* k_pages;              // [n_pages][Hkv][64][D]
  bf16* v_pages;              // [n_pages][Hkv][D][64]
  const int32_t* slot_map;    // [n_rows] page * 64 + row; -1: padding
  int n_rows, Hq, Hkv, n_pages;
  MropeAxes ax;
  int* status;
};
cudaError_t launch_mrope_append(const MropeAppendArgs& a, int D, cudaStream_t s);

// Attention of ragged chunks of rows over paged caches (csrc/attn_chunk.cu).
struct ChunkAttnArgs {
  bf16* out;                  // [n_rows][Hq][D]
  float* lse;                 // [n_rows][Hq] or NULL
  const int32_t* block_table; // [n_batch][max_pages]
  const int32_t* kv_len;      // [n_batch] slots, the new rows' included
  const int32_t* cu_rows;     // [n_batch + 1]
  const int32_t* n_noisy;     // [n_batch] or NULL (0): trailing rows that see every slot
  const int32_t* n_hidden;    // [n_batch] or NULL (0): leading slots that no row sees
  int n_batch, n_rows, n_pages, max_pages, Hq, Hkv;
  float scale_log2;
  void* workspace;
  int* status;
};
size_t attn_chunk_scratch_bytes(int P, int D);
// P: CTAs (one per SM).  q map: 3-D (D, Hq, rows), box (64, G, 128 / G).
cudaError_t launch_attn_chunk(const CUtensorMap& mapQ, const CUtensorMap& mapK, const CUtensorMap& mapV,
                              const ChunkAttnArgs& a, int D, int P, cudaStream_t s);

}  // namespace dvlm
