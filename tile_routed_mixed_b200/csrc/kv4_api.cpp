// Host side of the paged 4-bit cache's C ABI: argument checks, workspace layout
// and launches.  Allocates no memory.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "tilemix.h"
#include "tilemix_internal.h"
#include "tilemix_kv4.h"

namespace {

inline bool aligned(const void* p, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0;
}

// Whether two arrays share memory.
inline bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + m && b < a + n;
}

// log2 of a supported page size, or -1.
int page_shift(int page_size) {
  for (int sh = 4; sh <= 10; ++sh)
    if (page_size == 1 << sh) return sh;
  return -1;
}

// The pool's sizes; its pointers too where the call uses them.
int check_cache(const tilemix_kv4_cache& c, bool pointers) {
  if (c.d != 64 && c.d != 128) return TILEMIX_ERR_UNSUPPORTED;
  if ((c.group != 32 && c.group != 64 && c.group != 128) || c.group > c.d)
    return TILEMIX_ERR_UNSUPPORTED;
  if (c.dtype != TILEMIX_KV_FP16 && c.dtype != TILEMIX_KV_BF16) return TILEMIX_ERR_UNSUPPORTED;
  if (page_shift(c.page_size) < 0) return TILEMIX_ERR_UNSUPPORTED;
  if (c.num_pages < 1 || c.hk < 1 || c.hk > 32767 ||
      static_cast<long long>(c.num_pages) * c.page_size > 0x7fffffffLL)
    return TILEMIX_ERR_INVALID_ARG;
  if (!pointers) return TILEMIX_OK;
  if (!c.k_codes || !c.k_scale || !c.v_codes || !c.v_scale) return TILEMIX_ERR_INVALID_ARG;
  if (!aligned(c.k_codes, 16) || !aligned(c.k_scale, 16) || !aligned(c.v_codes, 16) ||
      !aligned(c.v_scale, 16))
    return TILEMIX_ERR_INVALID_ARG;
  return TILEMIX_OK;
}

tilemix::Kv4Pool pool_of(const tilemix_kv4_cache& c) {
  tilemix::Kv4Pool p;
  p.k_codes = c.k_codes;
  p.k_scale = static_cast<uint8_t*>(c.k_scale);
  p.v_codes = c.v_codes;
  p.v_scale = static_cast<uint8_t*>(c.v_scale);
  p.num_pages = c.num_pages;
  p.page_shift = page_shift(c.page_size);
  p.hk = c.hk;
  return p;
}

tilemix::Kv4Format format_of(const tilemix_kv4_cache& c) {
  return {c.d, c.group, c.dtype == TILEMIX_KV_BF16};
}

// A block table of nseq rows.
bool table_ok(int nseq, int max_pages) {
  return max_pages >= 1 && static_cast<long long>(nseq) * max_pages <= 0x7fffffffLL;
}

int check_attn(const tilemix_kv4_attn_args* a) {
  if (!a) return TILEMIX_ERR_INVALID_ARG;
  const int rc = check_cache(a->cache, false);
  if (rc != TILEMIX_OK) return rc;
  if (a->hq < 1 || a->hq % a->cache.hk != 0) return TILEMIX_ERR_INVALID_ARG;
  if (a->nseq < 0 || a->total_q < 0 || a->max_new < 1 || a->max_seqlen < 1 ||
      !table_ok(a->nseq, a->max_pages))
    return TILEMIX_ERR_INVALID_ARG;
  if (static_cast<long long>(a->total_q) * a->hq > 0x7fff0000LL) return TILEMIX_ERR_INVALID_ARG;
  if (!a->token_start && a->total_q < a->nseq) return TILEMIX_ERR_INVALID_ARG;
  if (!(a->softmax_scale >= 0.f) || std::isinf(a->softmax_scale)) return TILEMIX_ERR_INVALID_ARG;
  return TILEMIX_OK;
}

int current_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return 148;
  return sms;
}

struct AttnLayout {
  tilemix::Kv4AttnShape shape;
  size_t heads, parts, total;
};

// One state per warp (the unit that its tiles begin inside of) and two per
// CTA, whatever the batch; the shape follows the device and the column block.
AttnLayout attn_layout(const tilemix_kv4_attn_args* a) {
  AttnLayout w;
  const long long columns = static_cast<long long>(a->max_new) * (a->hq / a->cache.hk);
  w.shape = tilemix::kv4_attn_shape(current_sms(), columns, a->nseq, a->cache.hk, a->max_seqlen);
  const size_t state = static_cast<size_t>(w.shape.cols) * (a->cache.d + 2) * sizeof(float);
  w.heads = 0;
  w.parts = state * w.shape.ctas * w.shape.warps;
  w.total = (w.parts + state * w.shape.ctas * 2 + 255) / 256 * 256;
  return w;
}

}  // namespace

extern "C" {

TILEMIX_API int tilemix_page_plan(const tilemix_page_plan_args* a, void* stream) {
  if (!a) return TILEMIX_ERR_INVALID_ARG;
  if (a->nseq < 0 || a->num_pages < 1 || a->max_tokens < 0 || !table_ok(a->nseq, a->max_pages))
    return TILEMIX_ERR_INVALID_ARG;
  if (page_shift(a->page_size) < 0 || a->nseq > TILEMIX_PAGE_PLAN_MAX_SEQS)
    return TILEMIX_ERR_UNSUPPORTED;
  if (static_cast<long long>(a->num_pages) * a->page_size > 0x7fffffffLL)
    return TILEMIX_ERR_INVALID_ARG;
  if (!a->new_len || !a->seq_len || !a->block_table || !a->free_list || !a->free_count ||
      !a->token_start || (!a->slots && a->max_tokens > 0) || !a->granted)
    return TILEMIX_ERR_INVALID_ARG;
  tilemix::PagePlanParams p;
  p.new_len = a->new_len;
  p.seq_len = a->seq_len;
  p.block_table = a->block_table;
  p.free_list = a->free_list;
  p.free_count = a->free_count;
  p.token_start = a->token_start;
  p.slots = a->slots;
  p.granted = a->granted;
  p.nseq = a->nseq;
  p.max_pages = a->max_pages;
  p.num_pages = a->num_pages;
  p.page_shift = page_shift(a->page_size);
  p.max_tokens = a->max_tokens;
  // outputs are written while inputs are still read
  const size_t word = sizeof(int32_t), rows = word * a->nseq;
  const struct {
    const void* at;
    size_t bytes;
  } arrays[] = {{a->token_start, rows + word},
                {a->slots, word * a->max_tokens},
                {a->granted, rows},
                {a->new_len, rows},
                {a->seq_len, rows},
                {a->block_table, rows * a->max_pages},
                {a->free_list, word * a->num_pages},
                {a->free_count, word}};
  for (int i = 0; i < 7; ++i)
    for (int j = i + 1; j < 8; ++j)
      if (overlap(arrays[i].at, arrays[i].bytes, arrays[j].at, arrays[j].bytes))
        return TILEMIX_ERR_INVALID_ARG;
  if (tilemix::launch_page_plan(p, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return TILEMIX_ERR_CUDA;
  return TILEMIX_OK;
}

TILEMIX_API int tilemix_kv4_append(const tilemix_kv4_append_args* a, void* stream) {
  if (!a) return TILEMIX_ERR_INVALID_ARG;
  int rc = check_cache(a->cache, false);
  if (rc != TILEMIX_OK) return rc;
  const long long row = static_cast<long long>(a->cache.hk) * a->cache.d;
  if (a->n < 0 || static_cast<long long>(a->n) * row / 8 > 0x7fffffffLL)
    return TILEMIX_ERR_INVALID_ARG;
  if (a->n == 0) return TILEMIX_OK;
  if ((rc = check_cache(a->cache, true)) != TILEMIX_OK) return rc;
  if (!a->k || !a->v || !a->slots || !aligned(a->k, 16) || !aligned(a->v, 16))
    return TILEMIX_ERR_INVALID_ARG;
  if (a->k_stride < row || a->v_stride < row || a->k_stride % 8 != 0 || a->v_stride % 8 != 0)
    return TILEMIX_ERR_INVALID_ARG;
  tilemix::Kv4AppendParams p;
  p.pool = pool_of(a->cache);
  p.k = static_cast<const uint8_t*>(a->k);
  p.v = static_cast<const uint8_t*>(a->v);
  p.k_stride = a->k_stride * 2;
  p.v_stride = a->v_stride * 2;
  p.slots = a->slots;
  p.n = a->n;
  if (tilemix::launch_kv4_append(p, format_of(a->cache), static_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return TILEMIX_ERR_CUDA;
  return TILEMIX_OK;
}

TILEMIX_API int tilemix_kv4_gather(const tilemix_kv4_gather_args* a, void* stream) {
  if (!a) return TILEMIX_ERR_INVALID_ARG;
  int rc = check_cache(a->cache, false);
  if (rc != TILEMIX_OK) return rc;
  if (a->nseq < 0 || a->nseq > 65535 || a->rows < 0 || !table_ok(a->nseq, a->max_pages))
    return TILEMIX_ERR_INVALID_ARG;
  if (a->nseq == 0) return TILEMIX_OK;
  if ((rc = check_cache(a->cache, true)) != TILEMIX_OK) return rc;
  if (!a->block_table || !a->seq_len || !a->out_start) return TILEMIX_ERR_INVALID_ARG;
  if (a->rows > 0 && (!a->k || !a->v || !aligned(a->k, 16) || !aligned(a->v, 16)))
    return TILEMIX_ERR_INVALID_ARG;
  tilemix::Kv4GatherParams p;
  p.pool = pool_of(a->cache);
  p.block_table = a->block_table;
  p.seq_len = a->seq_len;
  p.out_start = a->out_start;
  p.k = static_cast<uint8_t*>(a->k);
  p.v = static_cast<uint8_t*>(a->v);
  p.nseq = a->nseq;
  p.max_pages = a->max_pages;
  p.rows = a->rows;
  const size_t out_bytes = static_cast<size_t>(a->rows) * a->cache.hk * a->cache.d * 2;
  if (overlap(a->k, out_bytes, a->v, out_bytes)) return TILEMIX_ERR_INVALID_ARG;
  if (tilemix::launch_kv4_gather(p, format_of(a->cache), static_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return TILEMIX_ERR_CUDA;
  return TILEMIX_OK;
}

TILEMIX_API int tilemix_kv4_attn_workspace_size(const tilemix_kv4_attn_args* a, size_t* bytes) {
  if (!a || !bytes) return TILEMIX_ERR_INVALID_ARG;
  const int rc = check_attn(a);
  if (rc != TILEMIX_OK) return rc;
  *bytes = attn_layout(a).total;
  return TILEMIX_OK;
}

TILEMIX_API int tilemix_kv4_attn(const tilemix_kv4_attn_args* a, void* stream) {
  int rc = check_attn(a);
  if (rc != TILEMIX_OK) return rc;
  if (a->nseq == 0 || a->total_q == 0) return TILEMIX_OK;
  if ((rc = check_cache(a->cache, true)) != TILEMIX_OK) return rc;
  if (!a->q || !a->o || !a->seq_len || !a->block_table || !a->sync || !aligned(a->q, 16) ||
      !aligned(a->o, 16))
    return TILEMIX_ERR_INVALID_ARG;
  const AttnLayout w = attn_layout(a);
  if (!a->workspace || a->workspace_bytes < w.total || !aligned(a->workspace, 256))
    return TILEMIX_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  tilemix::Kv4AttnParams p;
  p.pool = pool_of(a->cache);
  p.q = static_cast<const uint8_t*>(a->q);
  p.o = static_cast<uint8_t*>(a->o);
  p.lse = a->lse;
  p.token_start = a->token_start;
  p.seq_len = a->seq_len;
  p.block_table = a->block_table;
  p.granted = a->granted;
  p.heads = reinterpret_cast<float*>(ws + w.heads);
  p.parts = reinterpret_cast<float*>(ws + w.parts);
  p.sync = a->sync;
  p.nseq = a->nseq;
  p.total_q = a->total_q;
  p.max_pages = a->max_pages;
  p.hq = a->hq;
  p.group_q = a->hq / a->cache.hk;
  const float scale =
      a->softmax_scale > 0.f ? a->softmax_scale : 1.0f / std::sqrt(static_cast<float>(a->cache.d));
  p.scale_log2 = scale * 1.4426950408889634f;
  // a unit's O is written while others still read its rows of q
  const size_t q_bytes = static_cast<size_t>(a->total_q) * a->hq * a->cache.d * 2;
  const size_t lse_bytes = a->lse ? static_cast<size_t>(a->total_q) * a->hq * sizeof(float) : 0;
  if (overlap(a->q, q_bytes, a->o, q_bytes) || overlap(a->lse, lse_bytes, a->q, q_bytes) ||
      overlap(a->lse, lse_bytes, a->o, q_bytes))
    return TILEMIX_ERR_INVALID_ARG;
  if (tilemix::launch_kv4_attn(p, format_of(a->cache), w.shape,
                               static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return TILEMIX_ERR_CUDA;
  return TILEMIX_OK;
}

}  // extern "C"
