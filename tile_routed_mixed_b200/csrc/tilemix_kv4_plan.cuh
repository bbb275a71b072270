// Block tables and slot maps of one step (tilemix_page_plan).
//
// Every quantity is a prefix sum over the sequences: tokens added (where a
// sequence's slots start), pages needed (which free pages it takes) and pages
// returned (where they go on the stack).  The sums are taken once, in shared
// memory, by every CTA for itself; after that each returned page, each taken
// page and each slot is independent of all others and finds its sequence by
// bisection, so long prompts spread over all threads whatever their number.
//
// The work is a few hundred kilobytes at most: latency bounds it, not bytes.
// One launch does it all.  A cluster of CTAs shares the slots of large calls
// (its barrier orders the stack's writes before its reads); the tables' pages
// need no ordering against the slots, which compute their page from the stack.
// Included by tilemix_kv4.cu.
#pragma once

namespace tilemix {

constexpr int kPlanThreads = 512;
constexpr int kPlanCluster = 8;  // CTAs of a large call

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

struct Sums {
  long long grow, need, back;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {a.grow + b.grow, a.need + b.need, a.back + b.back};
}
__device__ __forceinline__ Sums shfl_up(const Sums& a, int by) {
  return {__shfl_up_sync(0xffffffffu, a.grow, by), __shfl_up_sync(0xffffffffu, a.need, by),
          __shfl_up_sync(0xffffffffu, a.back, by)};
}

// Exclusive sum over the block's threads; the total in *total.
__device__ __forceinline__ Sums block_exclusive(const Sums& mine, Sums* total) {
  __shared__ Sums warp_sum[kPlanThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums inc = mine;
#pragma unroll
  for (int by = 1; by < 32; by <<= 1) {
    const Sums up = shfl_up(inc, by);
    if (lane >= by) inc = inc + up;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  Sums base{0, 0, 0}, all{0, 0, 0};
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const Sums x = warp_sum[w];
    if (w < warp) base = base + x;
    all = all + x;
  }
  __syncthreads();
  *total = all;
  return {base.grow + inc.grow - mine.grow, base.need + inc.need - mine.need,
          base.back + inc.back - mine.back};
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
  plan::Sums mine{0, 0, 0};
  bool bad = free_in < 0 || free_in > p.num_pages;
  const long long F = min(max(free_in, 0), p.num_pages);
  const auto pages = [&](long long t) { return static_cast<int>((t + ps1) >> sh); };
  // tokens first: whether a sequence fits depends on where its tokens end
  for (int s = s0; s < s1; ++s) {
    const plan::Row r = plan::row_of(p.seq_len[s], __ldg(p.new_len + s), top);
    bad |= r.bad;
    mine.grow += r.grow;
    mine.back += pages(r.len) - pages(r.len - r.drop);
    len_s[s] = r.len;
  }
  plan::Sums total;
  plan::Sums before = plan::block_exclusive(mine, &total);
  const long long R = total.back;  // fewer than nseq * max_pages < 2^31
  long long end = before.grow, back = before.back;
  for (int s = s0; s < s1; ++s) {
    const int n = __ldg(p.new_len + s), len = len_s[s];
    const int grow = n > 0 ? n : 0;
    const int drop = plan::row_of(len, n, top).drop;
    const long long after = static_cast<long long>(len) + grow;
    end += grow;
    back += pages(len) - pages(len - drop);
    const bool fits = end <= p.max_tokens && after <= top;
    const int need = fits ? pages(after) - pages(len) : 0;
    mine.need += need;
    end_s[s] = plan::clamp31(end);
    back_s[s] = plan::clamp31(back);
    need_s[s] = need;
    flag_s[s] = fits;
  }
  plan::Sums total2;
  plan::Sums before2 = plan::block_exclusive({0, mine.need, 0}, &total2);
  const long long have = F + R;
  long long cum = before2.need, used = 0;
  for (int s = s0; s < s1; ++s) {
    const int need = need_s[s];
    cum += need;
    const bool ok = __ldg(p.new_len + s) <= 0 || (flag_s[s] && (need == 0 || cum <= have));
    if (ok) used += need;
    need_s[s] = plan::clamp31(cum);
    flag_s[s] = ok;
  }
  plan::Sums total3;
  plan::block_exclusive({0, used, 0}, &total3);
  used = total3.need;  // granted pages: a prefix of the needed ones
  __syncthreads();
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
  cudaError_t e = cudaFuncSetAttribute(page_plan_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return static_cast<int>(e);
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  // one CTA covers 2,048 slots in one sweep
  const int ctas = p.max_tokens > 4 * kPlanThreads ? kPlanCluster : 1;
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
