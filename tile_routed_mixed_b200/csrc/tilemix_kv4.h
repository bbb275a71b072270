// The paged 4-bit K/V cache: parameters of its kernels and their launchers
// (implemented in tilemix_kv4.cu; called by kv4_api.cpp).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace tilemix {

// Pool geometry shared by the kernels.  A row is one token's K or V of one KV
// head: d / 2 code bytes and d / group scales of two bytes, at row index
// (page * hk + kv) * page_size + offset of the code and scale arrays.
struct Kv4Pool {
  uint8_t* k_codes;
  uint8_t* k_scale;
  uint8_t* v_codes;
  uint8_t* v_scale;
  int num_pages, page_shift, hk;
};

struct PagePlanParams {
  const int32_t* new_len;
  int32_t* seq_len;
  int32_t* block_table;
  int32_t* free_list;
  int32_t* free_count;
  int32_t* token_start;
  int32_t* slots;
  int32_t* granted;
  int nseq, max_pages, num_pages, page_shift, max_tokens;
};

struct Kv4AppendParams {
  Kv4Pool pool;
  const uint8_t* k;
  const uint8_t* v;
  int64_t k_stride, v_stride;  // bytes
  const int32_t* slots;
  int n;
};

struct Kv4GatherParams {
  Kv4Pool pool;
  const int32_t* block_table;
  const int32_t* seq_len;
  const int32_t* out_start;
  uint8_t* k;
  uint8_t* v;
  int nseq, max_pages, rows;
};

struct Kv4AttnParams {
  Kv4Pool pool;
  const uint8_t* q;
  uint8_t* o;
  float* lse;
  const int32_t* token_start;
  const int32_t* seq_len;
  const int32_t* block_table;
  const int32_t* granted;  // or nullptr
  float* heads;        // workspace: partial states that a warp finishes mid-range
  float* parts;        // workspace: partial states of CTAs, two per CTA
  unsigned int* sync;  // arrivals of the CTAs that share a unit, by the unit's first CTA
  int nseq, total_q, max_pages, hq, group_q;  // group_q = hq / hk
  float scale_log2;    // softmax scale * log2(e)
};

// Formats a kernel is compiled for.
struct Kv4Format {
  int d, group;
  bool bf16;
};

int launch_page_plan(const PagePlanParams& p, cudaStream_t stream);
int launch_kv4_append(const Kv4AppendParams& p, const Kv4Format& f, cudaStream_t stream);
int launch_kv4_gather(const Kv4GatherParams& p, const Kv4Format& f, cudaStream_t stream);
// Attention launches: the most CTAs on this device (one per SM; sizes the
// workspace), those of this launch, warps of each, and columns of a block.
struct Kv4AttnShape {
  int ctas, grid, warps, cols;
};
Kv4AttnShape kv4_attn_shape(int sms, long long columns, long long nseq, int hk, long long keys);
int launch_kv4_attn(const Kv4AttnParams& p, const Kv4Format& f, const Kv4AttnShape& shape,
                    cudaStream_t stream);
int kv4_read_and_clear_status(unsigned int* status);

}  // namespace tilemix
