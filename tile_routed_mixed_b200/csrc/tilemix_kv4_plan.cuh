// Block tables and slot maps of one step (tilemix_page_plan).
//
// Every quantity is a prefix sum over the sequences: tokens added (where a
// sequence's slots start), pages needed (which free pages it takes) and pages
// returned (where they go on the stack).  The sums are taken once, in shared
// memory, by every CTA for itself; after that each returned page, each taken
// page and each slot is independent of all others and finds its sequence by
// bisection, so long prompts spread over all threads whatever their number.
//
// The work is a few hundred kilobytes at most: latency bounds it, not bytes (256
// sequences of one token 4.2 us, 125,000 slots of 64 prompts 7.2 us, their
// rollback 10 us).  One launch does it all.  A cluster of sixteen CTAs shares the
// slots of large calls (eight: 10.7 us; a cluster for 256 tokens: 4.6 us for 4.2);
// its barrier orders the stack's writes before its reads, and the slots need none
// against the tables, as they compute their page from the stack.
// Included by tilemix_kv4.cu.
#pragma once

namespace tilemix {

constexpr int kPlanThreads = 512;
constexpr int kPlanCluster = 16;  // CTAs of a large call

namespace plan {

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cluster_rank() {
  int r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Number of entries of the non-decreasing a[0 .. n) that are <= x.
__device__ __forceinline__ int count_le(const int* a, int n, int x) {
  int lo = 0;
  while (n > 0) {
    const int half = n >> 1;
    if (a[lo + half] <= x) {
      lo += half + 1;
      n -= half + 1;
    } else {
      n = half;
    }
  }
  return lo;
}

// Exclusive sums over the block's threads, and the totals.
template <class X>
__device__ __forceinline__ X block_exclusive(X mine, X* total) {
  __shared__ X warp_sum[kPlanThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  X upto = mine;
#pragma unroll
  for (int by = 1; by < 32; by <<= 1) {
    const X up = __shfl_up_sync(0xffffffffu, upto, by);
    if (lane >= by) upto += up;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  // every warp adds up the warps' sums for itself
  X all = lane < kPlanThreads / 32 ? warp_sum[lane] : X(0);
#pragma unroll
  for (int by = 1; by < 32; by <<= 1) {
    const X up = __shfl_up_sync(0xffffffffu, all, by);
    if (lane >= by) all += up;
  }
  *total = __shfl_sync(0xffffffffu, all, 31);
  const X before = __shfl_sync(0xffffffffu, all, max(warp - 1, 0));
  return (warp > 0 ? before : X(0)) + upto - mine;
}

__device__ __forceinline__ int clamp31(long long x) {
  return x > 0x7fffffffLL ? 0x7fffffff : static_cast<int>(x);
}

// A sequence's length and its new length as the plan reads them.
struct Row {
  int len, grow, drop;  // tokens held, added, dropped
  bool bad;             // the length lies outside the table
};
__device__ __forceinline__ Row row_of(int len, int n, long long top) {
  Row r;
  r.bad = len < 0 || len > top;
  r.len = len < 0 ? 0 : static_cast<int>(len > top ? top : len);
  r.grow = n > 0 ? n : 0;
  r.drop = n < 0 ? static_cast<int>(min(-static_cast<long long>(n), static_cast<long long>(r.len)))
                 : 0;
  return r;
}

}  // namespace plan

// Dynamic shared memory: five int arrays of nseq entries.
__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PagePlanParams p) {
  extern __shared__ int plan_smem[];
  int* len_s = plan_smem;          // tokens held
  int* end_s = len_s + p.nseq;     // tokens added up to and including s
  int* need_s = end_s + p.nseq;    // pages needed, likewise
  int* back_s = need_s + p.nseq;   // pages returned, likewise
  int* flag_s = back_s + p.nseq;   // granted
  const int sh = p.page_shift, ps1 = (1 << sh) - 1;
  // the last length a table row holds; positions stay inside an int
  const long long top = min(static_cast<long long>(p.max_pages) << sh, 0x7fffffffLL);
  const int tid = threadIdx.x;
  const int rank = plan::cluster_rank();
  const bool clustered = gridDim.x > 1;
  const int at = rank * kPlanThreads + tid, step = gridDim.x * kPlanThreads;

  const int per = (p.nseq + kPlanThreads - 1) / kPlanThreads;
  const int s0 = min(p.nseq, tid * per), s1 = min(p.nseq, s0 + per);
  const int free_in = *p.free_count;
  bool bad = free_in < 0 || free_in > p.num_pages;
  const long long F = min(max(free_in, 0), p.num_pages);
  const auto pages = [&](long long t) { return static_cast<int>((t + ps1) >> sh); };
  __shared__ int granted_pages;
  if (tid == 0) granted_pages = 0;
  // tokens first: whether a sequence fits depends on where its tokens end
  long long tokens_here = 0;
  int back_here = 0;  // all returned pages: fewer than nseq * max_pages < 2^31
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    const plan::Row r = plan::row_of(p.seq_len[s], __ldg(p.new_len + s), top);
    bad |= r.bad;
    tokens_here += r.grow;
    back_here += pages(r.len) - pages(r.len - r.drop);
    len_s[s] = r.len;
  }
  long long tokens;
  int returned;
  long long end = plan::block_exclusive(tokens_here, &tokens);
  int back = plan::block_exclusive(back_here, &returned);
  long long need_here = 0;
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    const plan::Row r = plan::row_of(len_s[s], __ldg(p.new_len + s), top);
    const long long after = static_cast<long long>(r.len) + r.grow;
    end += r.grow;
    back += pages(r.len) - pages(r.len - r.drop);
    const bool fits = end <= p.max_tokens && after <= top;
    const int need = fits ? pages(after) - pages(r.len) : 0;
    need_here += need;
    end_s[s] = plan::clamp31(end);
    back_s[s] = back;
    need_s[s] = need;
    flag_s[s] = fits;
  }
  long long needed;
  long long cum = plan::block_exclusive(need_here, &needed);
  const long long R = returned, have = F + R;
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    const int need = need_s[s];
    cum += need;
    const bool ok = __ldg(p.new_len + s) <= 0 || (flag_s[s] && (need == 0 || cum <= have));
    // pages granted are a prefix of those needed
    if (ok && need > 0) atomicMax(&granted_pages, static_cast<int>(cum));
    need_s[s] = plan::clamp31(cum);
    flag_s[s] = ok;
  }
  __syncthreads();
  const long long used = granted_pages;
  if (clustered) plan::cluster_sync();  // every CTA has read the lengths and the stack's height

  // returned pages onto the stack
  for (long long k = at; k < R; k += step) {
    const int s = plan::count_le(back_s, p.nseq, static_cast<int>(k));
    const int first = static_cast<int>(k) - (s > 0 ? back_s[s - 1] : 0);
    const int n = __ldg(p.new_len + s);
    const int keep = pages(len_s[s] - plan::row_of(len_s[s], n, top).drop);
    int32_t* entry = p.block_table + static_cast<size_t>(s) * p.max_pages + keep + first;
    const int page = *entry;
    *entry = -1;
    bad |= page < 0 || page >= p.num_pages;
    const long long place = have - 1 - k;
    if (place < p.num_pages)
      p.free_list[place] = page;
    else
      bad = true;
  }
  if (R > 0) {
    if (clustered)
      plan::cluster_sync();
    else
      __syncthreads();
  }
  // the k-th page taken
  const auto taken = [&](long long k) {
    const long long place = have - 1 - k;
    const int page = place < p.num_pages ? p.free_list[place] : -1;
    return page;
  };
  for (long long k = at; k < used; k += step) {
    const int s = plan::count_le(need_s, p.nseq, static_cast<int>(k));
    const int first = static_cast<int>(k) - (s > 0 ? need_s[s - 1] : 0);
    const int page = taken(k);
    bad |= page < 0 || page >= p.num_pages;
    p.block_table[static_cast<size_t>(s) * p.max_pages + pages(len_s[s]) + first] = page;
  }
  // slots, four tokens of a thread at a time
  const bool wide = (reinterpret_cast<uintptr_t>(p.slots) & 15) == 0;
  for (long long i0 = 4LL * at; i0 < p.max_tokens; i0 += 4LL * step) {
    int out[4];
    int s = plan::count_le(end_s, p.nseq, static_cast<int>(i0));
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long long i = i0 + u;
      out[u] = -1;
      if (i >= p.max_tokens) continue;
      while (s < p.nseq && end_s[s] <= i) ++s;
      if (s >= p.nseq || !flag_s[s]) continue;
      const int len = len_s[s];
      const long long pos = len + i - (s > 0 ? end_s[s - 1] : 0);
      const int j = static_cast<int>(pos >> sh), held = pages(len);
      const int page = j < held
                           ? p.block_table[static_cast<size_t>(s) * p.max_pages + j]
                           : taken((s > 0 ? need_s[s - 1] : 0) + static_cast<long long>(j - held));
      if (page < 0 || page >= p.num_pages)
        bad = true;
      else
        out[u] = (page << sh) + static_cast<int>(pos & ps1);
    }
    if (wide && i0 + 4 <= p.max_tokens)
      *reinterpret_cast<int4*>(p.slots + i0) = make_int4(out[0], out[1], out[2], out[3]);
    else
      for (int u = 0; u < 4 && i0 + u < p.max_tokens; ++u) p.slots[i0 + u] = out[u];
  }
  // lengths, offsets and grants, by the first CTA
  if (rank == 0) {
    for (int s = tid; s < p.nseq; s += kPlanThreads) {
      const int n = __ldg(p.new_len + s), len = len_s[s];
      const bool ok = flag_s[s];
      p.token_start[s + 1] = end_s[s];
      p.granted[s] = ok;
      p.seq_len[s] = n > 0 ? (ok ? len + n : len) : len - plan::row_of(len, n, top).drop;
    }
    if (tid == 0) {
      p.token_start[0] = 0;
      *p.free_count = static_cast<int>(min(have - used, static_cast<long long>(p.num_pages)));
    }
  }
  if (bad) atomicOr(&g_kv4_status, kStatusBadPages);
}

int launch_page_plan(const PagePlanParams& p, cudaStream_t stream) {
  const int smem = 5 * static_cast<int>(sizeof(int)) * p.nseq;
  // The limit belongs to the function, not to the call: every call sets the same
  // one, so that a small call of another thread takes nothing from a large one.
  cudaError_t e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       5 * static_cast<int>(sizeof(int)) * TILEMIX_PAGE_PLAN_MAX_SEQS);
  if (e != cudaSuccess) return static_cast<int>(e);
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  // one CTA covers 2,048 slots in one sweep
  const int ctas = p.max_tokens > 4 * kPlanThreads ? kPlanCluster : 1;
  if (ctas > 8 &&
      (e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) !=
          cudaSuccess)
    return static_cast<int>(e);
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, page_plan_kernel, p));
}

}  // namespace tilemix
