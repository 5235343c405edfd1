// blocks.hip -- block tables and slot maps from request lengths, and pages back to their pool.
// Included into engram_device.hip.
//
// A pool is a bitmap of free pages, so that pages come back in any order and from any number of
// workgroups with the same result, and the pages of a call are the lowest free ones.  The plan
// runs in one workgroup: three prefix sums share one scan (tokens and new blocks of the rows,
// free pages of the bitmap), after which every thread knows whether the call fits, and page k of
// the call is found from both ends by binary search: its bit in the bitmap, its row in the
// rows' sums.  What follows from that, a token's slot, is done by the same workgroup for few
// tokens and by a second launch for many.

namespace engram {

constexpr int kPlanThreads = 1024;
constexpr int kPlanGranules = 8;      // counted pieces of the bitmap per thread
constexpr uint32_t kSat = 0x7FFFFFFFu;  // sums stop here instead of wrapping round

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) {
  const uint32_t s = a + b;  // both at most kSat: no wrap
  return s < kSat ? s : kSat;
}

// The largest i in [0, n) with pre[i] <= k (pre ascending, pre[0] <= k).
__device__ __forceinline__ int last_at_most(const uint32_t* pre, int n, uint32_t k) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= k)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Position of the r-th (from 0) set bit of w, r < popcount(w).
__device__ __forceinline__ int nth_bit(uint32_t w, uint32_t r) {
  int at = 0;
#pragma unroll
  for (int half = 16; half >= 1; half >>= 1) {
    const uint32_t low = (uint32_t)__popc(w & ((1u << half) - 1u));
    if (r >= low) {
      r -= low;
      w >>= half;
      at += half;
    }
  }
  return at;
}

// w without its n lowest set bits, n < 32.
__device__ __forceinline__ uint32_t without_lowest(uint32_t w, uint32_t n) {
  for (uint32_t i = 0; i < n; ++i) w &= w - 1u;
  return w;
}

// The bits of word w that stand for pages.
__device__ __forceinline__ uint32_t plan_mask(const PlanArgs& a, int w) {
  const int pages = a.num_pages - 32 * w;
  return pages >= 32 ? ~0u : (1u << pages) - 1u;
}

// Position and slot of token t, the (t - start)-th new one of a row with `past` tokens.
__device__ __forceinline__ void write_token(const PlanArgs& a, int t, int row, uint32_t past, uint32_t start) {
  const uint32_t pos = past + (uint32_t)t - start;
  const uint32_t block = pos / (uint32_t)a.page_size;
  const int32_t page = a.tables[row * a.table_ld + block];
  int64_t slot = -1;
  if (page >= 0 && page < a.num_pages)
    slot = (int64_t)page * a.page_size + (pos - block * (uint32_t)a.page_size);
  else
    latch_error(ENGRAM_E_PAGE_RANGE);
  if (a.positions != nullptr) a.positions[t] = (int32_t)pos;
  if (a.token_slots != nullptr) a.token_slots[t] = slot;
}

__device__ __forceinline__ void write_no_token(const PlanArgs& a, int t) {
  if (a.positions != nullptr) a.positions[t] = 0;
  if (a.token_slots != nullptr) a.token_slots[t] = -1;
}

__device__ __forceinline__ uint32_t blocks_of(uint32_t len, uint32_t page_size) {
  return len == 0 ? 0u : (len - 1u) / page_size + 1u;
}

// Dynamic LDS: cu [R + 1], first page [R], past [R], granule sums [granules].
__global__ __launch_bounds__(kPlanThreads) void block_plan_kernel(PlanArgs a) {
  extern __shared__ uint32_t plan_lds[];
  uint32_t* cu = plan_lds;
  uint32_t* first = cu + a.R + 1;
  uint32_t* past = first + a.R;
  uint32_t* granule = past + a.R;
  __shared__ uint32_t wave_sum[3][kPlanThreads / 64];
  __shared__ int bad_row;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t P = (uint32_t)a.page_size;
  const int words = (a.num_pages + 31) / 32;
  if (tid == 0) bad_row = 0;
  __syncthreads();

  // this thread's rows, and its words of the bitmap
  const int per = (a.R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = tid * per, r1 = min(a.R, r0 + per);
  uint32_t tokens = 0, pages = 0;
  bool bad = false;
  for (int r = r0; r < r1; ++r) {
    const int32_t p = a.past[r], n = a.fresh[r];
    past[r] = (uint32_t)p;
    if (p < 0 || n < 0 || (int64_t)p + n > (int64_t)a.max_blocks * P) {
      bad = true;
      continue;
    }
    tokens = sat_add(tokens, (uint32_t)n);
    pages = sat_add(pages, blocks_of((uint32_t)(p + n), P) - blocks_of((uint32_t)p, P));
  }
  if (bad) bad_row = 1;
  uint32_t in_granule[kPlanGranules];
  uint32_t free_pages = 0;
  const int64_t w0 = (int64_t)tid * kPlanGranules * a.granule_words;
#pragma unroll
  for (int g = 0; g < kPlanGranules; ++g) {
    in_granule[g] = 0;
    for (int i = 0; i < a.granule_words; ++i) {
      const int64_t w = w0 + (int64_t)g * a.granule_words + i;
      if (w < words) in_granule[g] += (uint32_t)__popc(a.free[w] & plan_mask(a, (int)w));
    }
    free_pages += in_granule[g];
  }

  // one scan of all three
  uint32_t t_in = tokens, p_in = pages, f_in = free_pages;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t t = (uint32_t)__shfl_up((int)t_in, off, 64);
    const uint32_t p = (uint32_t)__shfl_up((int)p_in, off, 64);
    const uint32_t f = (uint32_t)__shfl_up((int)f_in, off, 64);
    if (lane >= off) {
      t_in = sat_add(t_in, t);
      p_in = sat_add(p_in, p);
      f_in += f;
    }
  }
  if (lane == 63) {
    wave_sum[0][wave] = t_in;
    wave_sum[1][wave] = p_in;
    wave_sum[2][wave] = f_in;
  }
  __syncthreads();
  uint32_t t_before = 0, p_before = 0, f_before = 0, t_all = 0, p_all = 0, f_all = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    if (w == wave) {
      t_before = t_all;
      p_before = p_all;
      f_before = f_all;
    }
    t_all = sat_add(t_all, wave_sum[0][w]);
    p_all = sat_add(p_all, wave_sum[1][w]);
    f_all += wave_sum[2][w];
  }
  bool fits = bad_row == 0 && t_all <= (uint32_t)a.T;
  if (!fits) {
    if (tid == 0) latch_error(ENGRAM_E_SEQLENS);
  } else if (p_all > f_all) {
    fits = false;
    if (tid == 0) latch_error(ENGRAM_E_PAGES);
  }
  if (!fits) {
    t_all = 0;
    p_all = 0;
  }

  // (below kSat every partial sum is exact)
  uint32_t at = t_before + t_in - tokens, page_at = p_before + p_in - pages;
  for (int r = r0; r < r1; ++r) {
    const uint32_t p = past[r];
    const uint32_t n = fits ? (uint32_t)a.fresh[r] : 0u;
    if (!fits) at = page_at = 0;
    cu[r] = at;
    first[r] = page_at;
    a.cu_seqlens[r] = (int32_t)at;
    if (a.seq_start != nullptr) a.seq_start[r] = p == 0 ? 1 : 0;
    if (a.lens != nullptr) a.lens[r] = (int32_t)(p + n);
    at += n;
    page_at += blocks_of(p + n, P) - blocks_of(p, P);
  }
  if (tid == 0) {
    cu[a.R] = t_all;
    a.cu_seqlens[a.R] = (int32_t)t_all;
  }
  const uint32_t free_at = f_before + f_in - free_pages;
  uint32_t sum = free_at;
#pragma unroll
  for (int g = 0; g < kPlanGranules; ++g) {
    granule[tid * kPlanGranules + g] = sum;
    sum += in_granule[g];
  }
  __syncthreads();

  for (uint32_t k = tid; k < p_all; k += kPlanThreads) {
    const int g = last_at_most(granule, kPlanThreads * kPlanGranules, k);
    uint32_t left = k - granule[g];
    int w = g * a.granule_words;
    uint32_t word = a.free[w] & plan_mask(a, w);
    for (uint32_t c = (uint32_t)__popc(word); left >= c; c = (uint32_t)__popc(word)) {
      left -= c;
      ++w;
      word = a.free[w] & plan_mask(a, w);
    }
    const int row = last_at_most(first, a.R, k);
    a.tables[row * a.table_ld + blocks_of(past[row], P) + (k - first[row])] = 32 * w + nth_bit(word, left);
  }
  __syncthreads();  // the tables are written, and the bitmap is read: it may be written now

  if (p_all > 0 || a.free_out != a.free) {
    uint32_t before = free_at;
    const int64_t w1 = min((int64_t)words, w0 + (int64_t)kPlanGranules * a.granule_words);
    for (int64_t w = w0; w < w1 && (before < p_all || a.free_out != a.free); ++w) {
      const uint32_t word = a.free[w], mine = word & plan_mask(a, (int)w);
      const uint32_t c = (uint32_t)__popc(mine);
      uint32_t out = word;
      if (before < p_all)
        out = before + c <= p_all ? word & ~mine : (word & ~mine) | without_lowest(mine, p_all - before);
      a.free_out[w] = out;
      before += c;
    }
  }
  if (!a.tokens_here) return;
  for (int t = tid; t < a.T; t += kPlanThreads) {
    if ((uint32_t)t >= t_all) {
      write_no_token(a, t);
      continue;
    }
    const int row = last_at_most(cu, a.R, (uint32_t)t);
    write_token(a, t, row, past[row], cu[row]);
  }
}

// Positions and slots of many tokens, from the sums that block_plan_kernel left in cu_seqlens.
__global__ __launch_bounds__(256) void block_tokens_kernel(PlanArgs a) {
  const uint32_t* cu = reinterpret_cast<const uint32_t*>(a.cu_seqlens);
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= a.T) return;
  if (a.R == 0 || (uint32_t)t >= cu[a.R]) {
    write_no_token(a, t);
    return;
  }
  const int row = last_at_most(cu, a.R, (uint32_t)t);
  const uint32_t start = cu[row];
  uint32_t past = (uint32_t)a.past[row];
  if (a.lens == a.past) past -= cu[row + 1] - start;  // the lengths stand there by now
  write_token(a, t, row, past, start);
}

// Tokens up to which one workgroup does it all.
constexpr int kPlanTokensHere = 4096;

hipError_t launch_block_plan(const PlanArgs& args, hipStream_t stream) {
  (void)hipGetLastError();  // drop a stale error another library left on this thread
  PlanArgs a = args;
  const int words = (a.num_pages + 31) / 32;
  a.granule_words = std::max(1, (words + kPlanThreads * kPlanGranules - 1) / (kPlanThreads * kPlanGranules));
  a.tokens_here = a.T <= kPlanTokensHere;
  const int lds = 4 * (3 * a.R + 1 + kPlanThreads * kPlanGranules);
  static std::atomic<uint64_t> done{0};
  hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(block_plan_kernel), 4 * (3 * kPlanMaxRows + 1 + kPlanThreads * kPlanGranules), done);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(block_plan_kernel, dim3(1), dim3(kPlanThreads), lds, stream, a);
  e = hipGetLastError();
  if (e != hipSuccess || a.tokens_here) return e;
  hipLaunchKernelGGL(block_tokens_kernel, dim3((unsigned)(((int64_t)a.T + 255) / 256)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Pages back to the pool, a workgroup a row.  Setting a bit twice is setting it once, so rows
// that share pages need no order.
__global__ __launch_bounds__(256) void block_release_kernel(ReleaseArgs a) {
  const int row = blockIdx.x;
  if (a.flags[row] == 0) return;
  const int32_t len = a.lens[row];
  if (len < 0 || len > (int64_t)a.max_blocks * a.page_size) {
    if (threadIdx.x == 0) latch_error(ENGRAM_E_SEQLENS);
    return;
  }
  const int blocks = (int)blocks_of((uint32_t)len, (uint32_t)a.page_size);
  for (int b = threadIdx.x; b < blocks; b += 256) {
    const int32_t page = a.tables[row * a.table_ld + b];
    if (page < 0 || page >= a.num_pages)
      latch_error(ENGRAM_E_PAGE_RANGE);
    else
      atomicOr(&a.free[page >> 5], 1u << (page & 31));
  }
}

hipError_t launch_block_release(const ReleaseArgs& a, hipStream_t stream) {
  (void)hipGetLastError();  // drop a stale error another library left on this thread
  if (a.R == 0) return hipSuccess;
  hipLaunchKernelGGL(block_release_kernel, dim3(a.R), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace engram
