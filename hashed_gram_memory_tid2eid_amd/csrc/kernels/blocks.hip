// blocks.hip -- block tables and slot maps from request lengths, and pages back to their pool.
// Included into engram_device.hip.
//
// A pool is a bitmap of free pages, so that pages come back in any order and from any number of
// workgroups with the same result, and the pages of a call are the lowest free ones.  The plan
// runs in one workgroup: the prefix sums of the rows' tokens and new blocks and of the bitmap's
// free pages share one scan, after which every thread knows whether the call fits, and the k-th
// page of the call is found by a binary search in the bitmap's sums, and its row by another in
// the rows'.  So does token t, many tokens in a launch of their own; where no row brings more
// than one token (decode) a row's thread writes its token, and up to 1,024 rows find their page,
// without a search for rows.  The call is a chain of latencies, not of bytes: what can be loaded is
// loaded before the scan and stays in registers.

namespace engram {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWords = 8;                           // words of the bitmap a thread loads at a time
// Up to so many pages are looked for one by one (4,096 of 64 rows 23.0 us, 6,144 28.6, 8,192 34.6,
// 65,536 203), more are handed out by the threads in whose words they are (28.1, 28.7, 27.6, 48.5).
constexpr uint32_t kPlanSearched = 6144;
constexpr uint32_t kSat = 0x7FFFFFFFu;                  // sums stop here instead of wrapping round

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) {
  const uint32_t s = a + b;  // both at most kSat: no wrap
  return s < kSat ? s : kSat;
}

// Inclusive sums over a row of 16 lanes, and over the wave.
__device__ __forceinline__ uint32_t row_scan(uint32_t v) {
  v = sat_add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false));  // row_shr:1
  v = sat_add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false));
  v = sat_add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false));
  return sat_add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false));
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v = row_scan(v);
  v = sat_add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));  // row_bcast:15
  return sat_add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));  // row_bcast:31
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

// The bits of word w that stand for pages (none where w is past the bitmap).
__device__ __forceinline__ uint32_t plan_mask(const PlanArgs& a, int64_t w) {
  const int64_t pages = a.num_pages - 32 * w;
  return pages >= 32 ? ~0u : pages <= 0 ? 0u : (1u << pages) - 1u;
}

// Free pages in words w .. w + kPlanWords - 1 as loaded.
__device__ __forceinline__ uint32_t count_words(const PlanArgs& a, int64_t w, int64_t words, const uint32_t* v) {
  uint32_t sum = 0;
  if (w + kPlanWords < words) {
#pragma unroll
    for (int i = 0; i < kPlanWords; ++i) sum += (uint32_t)__popc(v[i]);
  } else if (w < words) {
#pragma unroll
    for (int i = 0; i < kPlanWords; ++i) sum += (uint32_t)__popc(v[i] & plan_mask(a, w + i));
  }
  return sum;
}

// Words w .. w + kPlanWords - 1 of the bitmap as they are; 0 past it.
typedef uint32_t words_t __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ void load_words(const PlanArgs& a, int64_t w, int64_t words, uint32_t* out) {
  if (w + kPlanWords <= words) {
#pragma unroll
    for (int i = 0; i < kPlanWords; i += 4) {
      const words_t v = *reinterpret_cast<const words_t*>(a.free + w + i);
      out[i] = v.x, out[i + 1] = v.y, out[i + 2] = v.z, out[i + 3] = v.w;
    }
  } else if (w < words) {
#pragma unroll
    for (int i = 0; i < kPlanWords; ++i) out[i] = w + i < words ? a.free[w + i] : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < kPlanWords; ++i) out[i] = 0u;
  }
}

// The page of rank k among the free ones, k < their number: sums [count] are those before every
// stretch of `stretch` words.
__device__ __forceinline__ int find_page(const PlanArgs& a, const uint32_t* sums, int count, int64_t stretch,
                                         int64_t words, uint32_t k) {
  const int at = last_at_most(sums, count, k);
  uint32_t left = k - sums[at];
  for (int64_t w = at * stretch;; w += kPlanWords) {
    uint32_t v[kPlanWords];
    load_words(a, w, words, v);
#pragma unroll
    for (int i = 0; i < kPlanWords; ++i) {
      const uint32_t word = v[i] & plan_mask(a, w + i), n = (uint32_t)__popc(word);
      if (left < n) return (int)(32 * (w + i)) + nth_bit(word, left);
      left -= n;
    }
  }
}

// x / page_size, from mulhi(x, floor((2^32 - 1) / page_size)): that or one less.  (One CU does the
// whole call, so instructions count: a division of the compiler's takes some 30.)
__device__ __forceinline__ uint32_t block_at(const PlanArgs& a, uint32_t x) {
  const uint32_t q = __umulhi(x, a.page_inverse);
  return x - q * (uint32_t)a.page_size >= (uint32_t)a.page_size ? q + 1u : q;
}
// Blocks that a length takes (length + page_size < 2^32).
__device__ __forceinline__ uint32_t blocks_in(const PlanArgs& a, uint32_t len) {
  return block_at(a, len + (uint32_t)a.page_size - 1u);
}

// The slot of a token at `pos` of a row, on `page`.
__device__ __forceinline__ int64_t token_slot(const PlanArgs& a, int32_t page, uint32_t offset) {
  if (page >= 0 && page < a.num_pages) return (int64_t)page * a.page_size + offset;
  latch_error(ENGRAM_E_PAGE_RANGE);
  return -1;
}

// Position and slot of token t, the (t - start)-th new one of a row with `past` tokens.
__device__ __forceinline__ void write_token(const PlanArgs& a, int t, int row, uint32_t past, uint32_t start) {
  const uint32_t pos = past + (uint32_t)t - start;
  const uint32_t block = block_at(a, pos);
  const int32_t page = a.tables[row * a.table_ld + block];
  if (a.positions != nullptr) a.positions[t] = (int32_t)pos;
  a.token_slots[t] = token_slot(a, page, pos - block * (uint32_t)a.page_size);
}

__device__ __forceinline__ void write_no_token(const PlanArgs& a, int t) {
  if (a.positions != nullptr) a.positions[t] = 0;
  a.token_slots[t] = -1;
}

// The bitmap is TILES tiles of kPlanThreads * stretch words; thread i counts stretch i of each.
// Dynamic LDS: free pages before every stretch [TILES][kPlanThreads], then cu, first page and
// past of the rows [R] each.  A thread has up to ROWS rows, kPlanThreads apart, whose sums are
// scanned as the tiles' are, one after another.
template <int TILES, int ROWS>
__global__ __launch_bounds__(kPlanThreads) void block_plan_kernel(PlanArgs a) {
  extern __shared__ uint32_t plan_lds[];
  uint32_t* sums = plan_lds;
  uint32_t* cu = sums + TILES * kPlanThreads;
  uint32_t* first = cu + a.R;
  uint32_t* past = first + a.R;
  constexpr int kFree = 2 * ROWS, kSums = kFree + TILES;
  __shared__ uint32_t wave_sum[kSums + 1][kPlanThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t P = (uint32_t)a.page_size;
  const uint32_t most = (uint32_t)a.max_blocks * P;  // tokens a row can hold
  const int64_t words = (a.num_pages + 31) / 32, stretch = a.stretch;

  // this thread's rows, and its words of the bitmap
  uint32_t p[ROWS], n[ROWS], need[ROWS];
  int32_t page[ROWS];
  uint32_t in[kSums];
  uint32_t kept[TILES][kPlanWords];  // the last words of each stretch: all of them where it has no more
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int row = r * kPlanThreads + tid;
    p[r] = row < a.R ? (uint32_t)a.past[row] : 0u;
    n[r] = row < a.R ? (uint32_t)a.fresh[row] : 0u;
  }
#pragma unroll
  for (int j = 0; j < TILES; ++j) {
    in[kFree + j] = 0;
    const int64_t w0 = ((int64_t)j * kPlanThreads + tid) * stretch;
    for (int64_t w = w0; w < w0 + stretch; w += kPlanWords) {
      load_words(a, w, words, kept[j]);
      in[kFree + j] += count_words(a, w, words, kept[j]);
    }
  }
  bool longer = false;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    page[r] = -1;
    need[r] = 0;
    in[r] = in[ROWS + r] = 0;
    if (n[r] == 0 && (int32_t)p[r] >= 0 && p[r] <= most) continue;
    if ((int32_t)(p[r] | n[r]) < 0 || p[r] + n[r] > most) {
      in[r] = kSat;  // more tokens than any call has places for
      continue;
    }
    longer |= n[r] > 1;
    const uint32_t block = block_at(a, p[r]), have = block * P < p[r] ? block + 1u : block;
    need[r] = blocks_in(a, p[r] + n[r]) - have;
    in[r] = n[r];
    in[ROWS + r] = need[r];
    if (have > block && a.tokens_here) page[r] = a.tables[((int64_t)r * kPlanThreads + tid) * a.table_ld + block];
  }

  // one scan of all of them
  uint32_t before[kSums], all[kSums];
#pragma unroll
  for (int i = 0; i < kSums; ++i) {
    before[i] = wave_scan(in[i]);
    if (lane == 63) wave_sum[i][wave] = before[i];
  }
  const bool wave_longer = __ballot(longer) != 0;
  if (lane == 63) wave_sum[kSums][wave] = wave_longer;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSums; ++i) {
    const uint32_t of_wave = wave_sum[i][lane & 15];
    const uint32_t to = row_scan(of_wave);
    all[i] = (uint32_t)__builtin_amdgcn_readlane((int)to, 15);
    before[i] = before[i] - in[i] + (uint32_t)__builtin_amdgcn_readlane((int)(to - of_wave), wave);
  }
  const bool single = __ballot(wave_sum[kSums][lane & 15] != 0) == 0;
  const bool alone = single && ROWS == 1;  // every thread finds its own row's page
  uint32_t num_tokens = 0, num_new = 0, num_free = 0;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    before[r] += num_tokens;
    num_tokens = sat_add(num_tokens, all[r]);
    before[ROWS + r] += num_new;
    num_new = sat_add(num_new, all[ROWS + r]);
  }
#pragma unroll
  for (int j = 0; j < TILES; ++j) {
    before[kFree + j] += num_free;
    num_free += all[kFree + j];
  }
  const bool fits = num_tokens <= (uint32_t)a.T && num_new <= num_free;
  if (!fits) {
    if (tid == 0) latch_error(num_tokens > (uint32_t)a.T ? ENGRAM_E_SEQLENS : ENGRAM_E_PAGES);
    num_tokens = num_new = 0;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) n[r] = need[r] = before[r] = before[ROWS + r] = 0;
  }

  // (sums are exact below kSat)
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int row = r * kPlanThreads + tid;
    if (row >= a.R) break;
    if (!alone) {
      cu[row] = before[r];
      first[row] = before[ROWS + r];
      past[row] = p[r];
    }
    a.cu_seqlens[row] = (int32_t)before[r];
    if (a.seq_start != nullptr) a.seq_start[row] = p[r] == 0 ? 1 : 0;
    if (a.lens != nullptr) a.lens[row] = (int32_t)(p[r] + n[r]);
  }
  if (tid == 0) a.cu_seqlens[a.R] = (int32_t)num_tokens;
  if (num_new > 0) {
#pragma unroll
    for (int j = 0; j < TILES; ++j) sums[j * kPlanThreads + tid] = before[kFree + j];
  }
  if (num_new > 0 || !alone) __syncthreads();

  if (alone) {
    if (need[0] > 0) {
      page[0] = find_page(a, sums, TILES * kPlanThreads, stretch, words, before[ROWS]);
      a.tables[tid * a.table_ld + block_at(a, p[0])] = page[0];
    }
  } else if (num_new <= kPlanSearched) {
    for (uint32_t k = tid; k < num_new; k += kPlanThreads) {
      const int row = last_at_most(first, a.R, k);
      a.tables[row * a.table_ld + blocks_in(a, past[row]) + (k - first[row])] =
          find_page(a, sums, TILES * kPlanThreads, stretch, words, k);
    }
  } else {
    // every thread hands out the pages of its own words, in order, and goes along the rows
#pragma unroll 1
    for (int j = 0; j < TILES; ++j) {
      const int64_t w0 = ((int64_t)j * kPlanThreads + tid) * stretch;
      uint32_t k = sums[j * kPlanThreads + tid];
      if (k >= num_new) break;
      int row = last_at_most(first, a.R, k);
      uint32_t next = row + 1 < a.R ? first[row + 1] : kSat;
      int32_t* entry = a.tables + row * a.table_ld + blocks_in(a, past[row]) + (k - first[row]);
#pragma unroll 1
      for (int64_t w = w0; w < w0 + stretch && w < words && k < num_new; ++w) {
        for (uint32_t mine = a.free[w] & plan_mask(a, w); mine != 0 && k < num_new; mine &= mine - 1u) {
          if (k >= next) {
            do {
              ++row;
              next = row + 1 < a.R ? first[row + 1] : kSat;
            } while (k >= next);
            entry = a.tables + row * a.table_ld + blocks_in(a, past[row]);
          }
          *entry++ = (int32_t)(32 * w) + __ffs(mine) - 1;
          ++k;
        }
      }
    }
  }
  if (num_new > 0) __syncthreads();  // tables are written, and the bitmap is read: it may be written now

  if (num_new > 0 || a.free_out != a.free) {
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      const int64_t w0 = ((int64_t)j * kPlanThreads + tid) * stretch;
      uint32_t ahead = before[kFree + j];  // free pages before the word
      for (int64_t w = w0; w < w0 + stretch && w < words; w += kPlanWords) {
        if (ahead >= num_new && a.free_out == a.free) break;
        if (stretch > kPlanWords) load_words(a, w, words, kept[j]);
        if (ahead < num_new) {
#pragma unroll
          for (int i = 0; i < kPlanWords; ++i) {
            const uint32_t mine = kept[j][i] & plan_mask(a, w + i), c = (uint32_t)__popc(mine);
            if (ahead < num_new)
              kept[j][i] = (kept[j][i] & ~mine) | (ahead + c <= num_new ? 0u : without_lowest(mine, num_new - ahead));
            ahead += c;
          }
        }
        if (w + kPlanWords <= words) {
#pragma unroll
          for (int i = 0; i < kPlanWords; i += 4)
            *reinterpret_cast<words_t*>(a.free_out + w + i) =
                words_t{kept[j][i], kept[j][i + 1], kept[j][i + 2], kept[j][i + 3]};
        } else {
#pragma unroll
          for (int i = 0; i < kPlanWords; ++i)
            if (w + i < words) a.free_out[w + i] = kept[j][i];
        }
      }
    }
  }
  if (!a.tokens_here) return;
  if (single) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (n[r] == 0) continue;
      const uint32_t block = block_at(a, p[r]);
      if (!alone && need[r] > 0) page[r] = a.tables[((int64_t)r * kPlanThreads + tid) * a.table_ld + block];
      if (a.positions != nullptr) a.positions[before[r]] = (int32_t)p[r];
      a.token_slots[before[r]] = token_slot(a, page[r], p[r] - block * P);
    }
    for (int t = (int)num_tokens + tid; t < a.T; t += kPlanThreads) write_no_token(a, t);
    return;
  }
  for (int t = tid; t < a.T; t += kPlanThreads) {
    if ((uint32_t)t >= num_tokens) {
      write_no_token(a, t);
      continue;
    }
    const int row = last_at_most(cu, a.R, (uint32_t)t);
    write_token(a, t, row, past[row], cu[row]);
  }
}

// Positions and slots of many tokens, from the sums that block_plan_kernel left in cu_seqlens.
constexpr int kTokenRows = 2048;  // up to so many rows' sums are searched in LDS
__global__ __launch_bounds__(256) void block_tokens_kernel(PlanArgs a) {
  __shared__ uint32_t near[kTokenRows];
  const uint32_t* cu = reinterpret_cast<const uint32_t*>(a.cu_seqlens);
  const int t = blockIdx.x * 256 + threadIdx.x;
  const uint32_t total = cu[a.R];
  if (a.R <= kTokenRows) {
    for (int r = threadIdx.x; r < a.R; r += 256) near[r] = cu[r];
    __syncthreads();
  }
  if (t >= a.T) return;
  if ((uint32_t)t >= total) {
    write_no_token(a, t);
    return;
  }
  const int row = a.R <= kTokenRows ? last_at_most(near, a.R, (uint32_t)t) : last_at_most(cu, a.R, (uint32_t)t);
  const uint32_t start = cu[row];
  uint32_t past = (uint32_t)a.past[row];
  if (a.lens == a.past) past -= cu[row + 1] - start;  // the lengths stand there by now
  write_token(a, t, row, past, start);
}

// One workgroup does it all for up to 4,096 tokens (64 rows: 9.5 us, two launches 9.3; 2,048 tokens
// 8.1 against 9.2, 8,192 tokens 12.8 against 9.4), or about a token a row (2,048 rows 12.8 against
// 17.4, 4,096 rows of 1M pages 15.3 against 18.8, 8,192 rows 22.6 against 24.6).
constexpr int kPlanTokensHere = 4096;

template <int TILES, int ROWS>
static hipError_t launch_plan_of(const PlanArgs& a, hipStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(block_plan_kernel<TILES, ROWS>),
                                          4 * (TILES + 3 * ROWS) * kPlanThreads, done);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((block_plan_kernel<TILES, ROWS>), dim3(1), dim3(kPlanThreads),
                     4 * (TILES * kPlanThreads + 3 * a.R), stream, a);
  return hipGetLastError();
}

hipError_t launch_block_plan(const PlanArgs& args, hipStream_t stream) {
  (void)hipGetLastError();  // drop a stale error another library left on this thread
  PlanArgs a = args;
  const int64_t words = ((int64_t)a.num_pages + 31) / 32;
  constexpr int64_t tile = (int64_t)kPlanThreads * kPlanWords;
  a.tokens_here = a.T <= std::max(kPlanTokensHere, a.R + 1024);
  a.page_inverse = 0xFFFFFFFFu / (uint32_t)a.page_size;
  a.stretch = kPlanWords * std::max<int64_t>(1, (words + 4 * tile - 1) / (4 * tile));
  // one tile up to 262,144 pages; four up to any number, whose stretches grow past 1,048,576
  // (4,096 rows: 14.9 us by 4 a thread, 17.1 by 8)
  hipError_t e;
  if (a.R <= kPlanThreads)
    e = words <= tile ? launch_plan_of<1, 1>(a, stream) : launch_plan_of<4, 1>(a, stream);
  else if (a.R <= 4 * kPlanThreads)
    e = words <= tile ? launch_plan_of<1, 4>(a, stream) : launch_plan_of<4, 4>(a, stream);
  else
    e = words <= tile ? launch_plan_of<1, 8>(a, stream) : launch_plan_of<4, 8>(a, stream);
  if (e != hipSuccess || a.tokens_here) return e;
  hipLaunchKernelGGL(block_tokens_kernel, dim3((unsigned)(((int64_t)a.T + 255) / 256)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Sets the bits of a wave's pages (-1: none).  Setting a bit twice is setting it once, so the
// order does not matter.  A lane first takes over the bits that the lanes behind it have for the
// same word, and only the first of a run sets them: pages that were taken together lie together.
__device__ __forceinline__ void free_pages(uint32_t* free, int32_t page, int lane) {
  const int word = page >> 5;  // (-1 for none)
  uint32_t bits = page >= 0 ? 1u << (page & 31) : 0u;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int w = __shfl_down(word, off, 64);
    const uint32_t b = (uint32_t)__shfl_down((int)bits, off, 64);
    if (lane + off < 64 && w == word) bits |= b;
  }
  const int before = __shfl_up(word, 1, 64);
  if (page >= 0 && (lane == 0 || before != word)) atomicOr(&free[word], bits);
}

// Pages back to the pool, a workgroup a row.
__global__ __launch_bounds__(256) void block_release_kernel(ReleaseArgs a) {
  const int row = blockIdx.x;
  if (a.flags[row] == 0) return;
  const int32_t len = a.lens[row];
  if (len < 0 || len > (int64_t)a.max_blocks * a.page_size) {
    if (threadIdx.x == 0) latch_error(ENGRAM_E_SEQLENS);
    return;
  }
  const int blocks = (int)((len + a.page_size - 1LL) / a.page_size);
  for (int b0 = 0; b0 < blocks; b0 += 256) {
    const int b = b0 + threadIdx.x;
    int32_t page = -1;
    if (b < blocks) {
      page = a.tables[row * a.table_ld + b];
      if (page < 0 || page >= a.num_pages) {
        latch_error(ENGRAM_E_PAGE_RANGE);
        page = -1;
      }
    }
    free_pages(a.free, page, threadIdx.x & 63);
  }
}

hipError_t launch_block_release(const ReleaseArgs& a, hipStream_t stream) {
  (void)hipGetLastError();  // drop a stale error another library left on this thread
  if (a.R == 0) return hipSuccess;
  hipLaunchKernelGGL(block_release_kernel, dim3(a.R), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace engram
