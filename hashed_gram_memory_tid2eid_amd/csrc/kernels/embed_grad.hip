// embed_grad.hip -- the gradient of the lookup in embed.hip, by sorted tokens.  Included into
// engram_device.hip after embed.hip, whose helpers it uses.
//
//   grad[r][d] = scale * sum over the places (t, c) with ids[t][c] = r of dout[t][c seg_pitch + d]
//
// The places are sorted by row id (a stable radix sort, 8 bits a pass, over as many bits as
// the table's row count has; id -1 and ids outside the table sort behind every row), so a
// row's places are one run.  The sorted list is cut into chunks of `ch` places; a group of
// lanes owns one chunk and one range of columns, 8 per lane, and walks it with fp32 sums in
// registers.  A run inside a chunk is finished there and written once.  Runs that cross
// chunks leave partial rows: `head` (a run that came in from the chunk before) and `tail` (a
// run that starts here and goes on); a second level joins kJoin chunks the same way, and the
// last kernel joins what crosses those.  Nothing is added by atomics: the order of every sum
// follows the sorted places, so results repeat bit for bit.

namespace engram {

constexpr int kSortThreads = 256, kSortItems = 16, kSortTile = kSortThreads * kSortItems;
constexpr int kSegThreads = 256;
constexpr int kJoin = 32;        // chunks per second-level chunk
constexpr int kCountTile = 1024; // sorted places per workgroup of the run count

struct SortKArgs {
  const int32_t* ids;     // first pass: [T][ids_ld]
  const uint32_t* key_in; // later passes
  const uint32_t* pos_in;
  uint32_t* key_out;
  uint32_t* pos_out;
  uint32_t* hist;         // [256][blocks]
  uint32_t* total;        // [256]
  int64_t ids_ld;
  uint32_t n, rows, cols, blocks, shift;
  FastDiv div_cols;
};

// the sort key of place i: its row, or `rows` where it has none
template <bool FIRST, bool LATCH>
__device__ __forceinline__ uint32_t sort_key(const SortKArgs& a, uint32_t i) {
  if (!FIRST) return a.key_in[i];
  const uint32_t t = fdiv(i, a.div_cols);
  const int32_t id = a.ids[(int64_t)t * a.ids_ld + (i - t * a.cols)];
  if (id >= 0 && (uint32_t)id < a.rows) return (uint32_t)id;
  if (LATCH && id != -1) latch_error(ENGRAM_E_ROW_RANGE);
  return a.rows;
}

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortKArgs a) {
  __shared__ uint32_t cnt[256];
  cnt[threadIdx.x] = 0;
  __syncthreads();
  const uint32_t base = blockIdx.x * kSortTile;
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    const uint32_t at = base + i * kSortThreads + threadIdx.x;
    if (at < a.n) atomicAdd(&cnt[(sort_key<FIRST, true>(a, at) >> a.shift) & 255u], 1u);
  }
  __syncthreads();
  a.hist[threadIdx.x * a.blocks + blockIdx.x] = cnt[threadIdx.x];
}

// exclusive sum over the 256 threads of a workgroup; *all receives the total
__device__ __forceinline__ uint32_t scan256(uint32_t v, uint32_t* wsum, uint32_t* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t s = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)s, off, 64);
    if (lane >= off) s += o;
  }
  __syncthreads();  // the last call's readers are done with wsum
  if (lane == 63) wsum[wave] = s;
  __syncthreads();
  uint32_t before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < wave) before += wsum[w];
    sum += wsum[w];
  }
  *all = sum;
  return before + s - v;
}

// one workgroup per digit: its counts over the blocks become exclusive sums
__global__ __launch_bounds__(256) void sort_scan_kernel(SortKArgs a) {
  __shared__ uint32_t wsum[4];
  uint32_t* h = a.hist + (int64_t)blockIdx.x * a.blocks;
  uint32_t carry = 0;
  for (uint32_t b = 0; b < a.blocks; b += 256) {
    const uint32_t at = b + threadIdx.x;
    const uint32_t v = at < a.blocks ? h[at] : 0u;
    uint32_t all;
    const uint32_t ex = scan256(v, wsum, &all);
    if (at < a.blocks) h[at] = carry + ex;
    carry += all;
  }
  if (threadIdx.x == 0) a.total[blockIdx.x] = carry;
}

// Stable scatter of one pass: wave w owns places [1024 w, +1024) of the tile and ranks 64 of
// them at a time; the lanes with one digit find each other by 8 ballots.
template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(SortKArgs a) {
  __shared__ uint32_t cnt[4][256];
  __shared__ uint32_t wsum[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int w = 0; w < 4; ++w) cnt[w][tid] = 0;
  uint32_t all;
  const uint32_t digit_base = scan256(a.total[tid], wsum, &all) + a.hist[(int64_t)tid * a.blocks + blockIdx.x];
  __syncthreads();
  uint32_t key[kSortItems], pos[kSortItems], rank[kSortItems];
  const uint32_t base = blockIdx.x * kSortTile + wave * (64 * kSortItems);
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    const uint32_t at = base + i * 64 + lane;
    key[i] = at < a.n ? sort_key<FIRST, false>(a, at) : 0u;
    pos[i] = at < a.n ? (FIRST ? at : a.pos_in[at]) : 0u;
  }
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    const bool live = base + i * 64 + lane < a.n;
    const uint32_t d = (key[i] >> a.shift) & 255u;
    uint64_t peers = __ballot(live);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const bool bit = (d >> b) & 1u;
      const uint64_t m = __ballot(bit);
      peers &= bit ? m : ~m;
    }
    const uint32_t below = (uint32_t)__popcll(peers & ((1ull << lane) - 1ull));
    const uint32_t before = cnt[wave][d];
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
    if (live && below == 0) cnt[wave][d] = before + (uint32_t)__popcll(peers);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    rank[i] = before + below;
  }
  __syncthreads();
  uint32_t run = digit_base;  // thread = digit: first output place of each wave's part
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t c = cnt[w][tid];
    cnt[w][tid] = run;
    run += c;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    if (base + i * 64 + lane >= a.n) continue;
    const uint32_t to = cnt[wave][(key[i] >> a.shift) & 255u] + rank[i];
    a.key_out[to] = key[i];
    a.pos_out[to] = pos[i];
  }
}

// ---- runs of the sorted list (sparse gradients name their rows) -------------------

struct RunKArgs {
  const uint32_t* key;
  uint32_t n, rows, ch, tiles;
  uint32_t* chunk_runs;  // runs that start in the chunk's tile before the chunk
  uint32_t* tile_runs;   // runs per tile, then exclusive sums
  int32_t* unique;
  int32_t* count;
};

__global__ __launch_bounds__(256) void run_count_kernel(RunKArgs a) {
  __shared__ uint32_t wsum[4];
  const uint32_t i0 = blockIdx.x * kCountTile + threadIdx.x * 4;
  uint32_t c = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t i = i0 + e;
    if (i >= a.n) break;
    a.unique[i] = -1;
    const uint32_t k = a.key[i];
    if (k < a.rows && (i == 0 || a.key[i - 1] != k)) ++c;
  }
  uint32_t all;
  const uint32_t ex = scan256(c, wsum, &all);
  if (i0 < a.n && i0 % a.ch == 0) a.chunk_runs[i0 / a.ch] = ex;
  if (threadIdx.x == 0) a.tile_runs[blockIdx.x] = all;
}

__global__ __launch_bounds__(256) void run_scan_kernel(RunKArgs a) {
  __shared__ uint32_t wsum[4];
  uint32_t carry = 0;
  for (uint32_t b = 0; b < a.tiles; b += 256) {
    const uint32_t at = b + threadIdx.x;
    const uint32_t v = at < a.tiles ? a.tile_runs[at] : 0u;
    uint32_t all;
    const uint32_t ex = scan256(v, wsum, &all);
    if (at < a.tiles) a.tile_runs[at] = carry + ex;
    carry += all;
  }
  if (threadIdx.x == 0) *a.count = (int32_t)carry;
}

// ---- sums over the runs ------------------------------------------------------------

struct SegKArgs {
  const uint32_t* key;
  const uint32_t* pos;
  const void* dout;
  void* grad;
  float* head;    // [chunks][pdim]
  float* tail;
  float* head2;   // [chunks2][pdim]
  float* tail2;
  const uint32_t* chunk_runs;
  const uint32_t* tile_runs;
  int32_t* unique;
  int64_t dout_ld, seg_pitch, grad_ld;
  uint32_t n, rows, cols, ch, chunks, chunks2;
  int32_t dim, pdim, mode;
  float scale;
  int32_t dout_vec, grad_vec;
  uint32_t group_shift;  // log2 of the lanes per group
  FastDiv div_cols;
};

struct SegPlace {
  uint32_t unit;  // the chunk this group owns
  int32_t col;    // the lane's first column
};

__device__ __forceinline__ SegPlace seg_place(const SegKArgs& a) {
  const uint32_t lane = threadIdx.x & ((1u << a.group_shift) - 1u);
  SegPlace p;
  p.unit = (blockIdx.x << (8 - a.group_shift)) + (threadIdx.x >> a.group_shift);
  p.col = (int32_t)(((blockIdx.y << a.group_shift) + lane) * 8);
  return p;
}

// runs that start before sorted place i, the first of its chunk
__device__ __forceinline__ uint32_t runs_before(const SegKArgs& a, uint32_t i) {
  return a.tile_runs[i / kCountTile] + a.chunk_runs[i / a.ch];
}

template <bool GRAD_F32>
__device__ __forceinline__ void write_row(const SegKArgs& a, uint32_t key, uint32_t run, int32_t col, const float* acc) {
  const int n = min(8, a.dim - col);
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = acc[i] * a.scale;
  const bool sparse = a.mode == ENGRAM_GRAD_SPARSE;
  const int64_t at = (int64_t)(sparse ? run : key) * a.grad_ld + col;
  if (sparse && col == 0) a.unique[run] = (int32_t)key;
  if (a.mode == ENGRAM_GRAD_ACCUMULATE) {
    float old[8];
    load_chunk8<GRAD_F32>(a.grad, at, n, a.grad_vec != 0, old);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += old[i];
  }
  store_chunk8<GRAD_F32>(a.grad, at, n, a.grad_vec != 0, f);
}

__device__ __forceinline__ void put_partial(float* to, const SegKArgs& a, uint32_t unit, int32_t col, const float* acc) {
  f32x4* p = reinterpret_cast<f32x4*>(to + (int64_t)unit * a.pdim + col);
  p[0] = f32x4{acc[0], acc[1], acc[2], acc[3]};
  p[1] = f32x4{acc[4], acc[5], acc[6], acc[7]};
}

__device__ __forceinline__ void add_partial(const float* from, const SegKArgs& a, uint32_t unit, int32_t col, float* acc) {
  const f32x4* p = reinterpret_cast<const f32x4*>(from + (int64_t)unit * a.pdim + col);
  const f32x4 lo = p[0], hi = p[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[i] += lo[i];
    acc[4 + i] += hi[i];
  }
}

__device__ __forceinline__ void clear8(float* acc) {
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
}

template <bool DOUT_F32, bool GRAD_F32>
__global__ __launch_bounds__(kSegThreads) void segment_sum_kernel(SegKArgs a) {
  constexpr int U = 4;  // rows in flight per lane
  const SegPlace p = seg_place(a);
  if (p.unit >= a.chunks || p.col >= a.dim) return;
  const uint32_t i0 = p.unit * a.ch, i1 = min(a.n, i0 + a.ch);
  uint32_t cur = a.key[i0];
  if (cur >= a.rows) return;
  bool started = i0 == 0 || a.key[i0 - 1] != cur;
  uint32_t run = 0;
  if (a.mode == ENGRAM_GRAD_SPARSE) run = runs_before(a, i0) - (started ? 0u : 1u);
  float acc[8];
  clear8(acc);
  bool done = false;
  for (uint32_t i = i0; i < i1 && !done; i += U) {
    uint32_t k[U];
    float f[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool live = i + u < i1;
      k[u] = live ? a.key[i + u] : a.rows;
      clear8(f[u]);
      if (k[u] < a.rows) {
        const uint32_t pos = a.pos[i + u];
        const uint32_t t = fdiv(pos, a.div_cols);
        // columns up to the next multiple of 8 lie in the segment when it starts on 16 bytes
        load_chunk8<DOUT_F32>(a.dout, (int64_t)t * a.dout_ld + (int64_t)(pos - t * a.cols) * a.seg_pitch + p.col,
                              a.dout_vec ? 8 : min(8, a.dim - p.col), a.dout_vec != 0, f[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= i1 || done) continue;
      if (k[u] != cur) {
        if (started) write_row<GRAD_F32>(a, cur, run, p.col, acc);
        else put_partial(a.head, a, p.unit, p.col, acc);
        clear8(acc);
        started = true;
        cur = k[u];
        ++run;
        if (cur >= a.rows) {
          done = true;
          continue;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += f[u][e];
    }
  }
  if (done) return;
  const bool goes_on = i1 < a.n && a.key[i1] == cur;
  if (!started) put_partial(a.head, a, p.unit, p.col, acc);
  else if (goes_on) put_partial(a.tail, a, p.unit, p.col, acc);
  else write_row<GRAD_F32>(a, cur, run, p.col, acc);
}

// whether the run of place i's left neighbour goes on at i (i > 0)
__device__ __forceinline__ bool linked(const SegKArgs& a, uint32_t i) {
  return i < a.n && a.key[i] < a.rows && a.key[i - 1] == a.key[i];
}

// the run index that a run reaching place i (the first of a chunk) from before has
__device__ __forceinline__ uint32_t run_into(const SegKArgs& a, uint32_t i) {
  return a.mode == ENGRAM_GRAD_SPARSE ? runs_before(a, i) - 1u : 0u;
}

// second level: one group per kJoin chunks
template <bool GRAD_F32>
__global__ __launch_bounds__(kSegThreads) void segment_join_kernel(SegKArgs a) {
  const SegPlace p = seg_place(a);
  if (p.unit >= a.chunks2 || p.col >= a.dim) return;
  const uint32_t c0 = p.unit * kJoin, c1 = min(a.chunks, c0 + kJoin);
  float acc[8];
  clear8(acc);
  bool in = c0 > 0 && linked(a, c0 * a.ch);
  bool started = false;  // whether the open run started in this unit
  for (uint32_t c = c0; c < c1; ++c) {
    const uint32_t i0 = c * a.ch, i1 = min(a.n, i0 + a.ch);
    const bool out = linked(a, i1);
    const bool whole = a.key[i0] == a.key[i1 - 1];
    if (in) {
      add_partial(a.head, a, c, p.col, acc);
      if (!(whole && out)) {  // the run ends in this chunk
        if (started) write_row<GRAD_F32>(a, a.key[i0], run_into(a, i0), p.col, acc);
        else put_partial(a.head2, a, p.unit, p.col, acc);
      }
    }
    if (out && !(whole && in)) {  // a run starts here and goes on
      clear8(acc);
      add_partial(a.tail, a, c, p.col, acc);
      started = true;
    }
    in = out;
  }
  if (!in) return;
  if (started) put_partial(a.tail2, a, p.unit, p.col, acc);
  else put_partial(a.head2, a, p.unit, p.col, acc);
}

// last level: the unit in which a run starts that leaves it adds what the following units hold
template <bool GRAD_F32>
__global__ __launch_bounds__(kSegThreads) void segment_finish_kernel(SegKArgs a) {
  const SegPlace p = seg_place(a);
  if (p.unit >= a.chunks2 || p.col >= a.dim) return;
  const uint32_t per = kJoin * a.ch;
  const uint32_t i0 = p.unit * per;
  if (a.n - i0 <= per) return;  // the last unit: nothing leaves it
  const uint32_t end = i0 + per;
  if (!linked(a, end)) return;
  const uint32_t k = a.key[end];
  if (p.unit > 0 && a.key[i0 - 1] == k) return;  // it started earlier
  float acc[8];
  clear8(acc);
  add_partial(a.tail2, a, p.unit, p.col, acc);
  uint32_t last = p.unit + 1;  // the unit in which the run ends
  while (a.n - last * per > per && a.key[(last + 1) * per] == k) ++last;
  for (uint32_t u = p.unit + 1; u <= last; ++u) add_partial(a.head2, a, u, p.col, acc);
  write_row<GRAD_F32>(a, k, run_into(a, end), p.col, acc);
}

template <bool F32>
__global__ __launch_bounds__(256) void zero_rows_kernel(void* grad, int64_t rows, int32_t dim, int64_t ld, int32_t vec,
                                                        uint32_t chunks) {
  const float z[8] = {};
  const int64_t total = rows * chunks;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / chunks;
    const int32_t col = (int32_t)(i - r * chunks) * 8;
    store_chunk8<F32>(grad, r * ld + col, min(8, dim - col), vec != 0, z);
  }
}

// ---- the workspace and the launches -------------------------------------------------

struct EmbedGradPlan {
  uint32_t n, ch, chunks, chunks2, blocks, tiles;
  int64_t pdim;
  int64_t key[2], pos[2], hist, total, chunk_runs, tile_runs, head, tail, head2, tail2, bytes;
};

static EmbedGradPlan embed_grad_plan(int64_t n, int32_t dim) {
  EmbedGradPlan p;
  p.n = (uint32_t)n;
  // places per chunk: few for short lists, so that they spread over the chip
  p.ch = n <= 32768 ? 8 : 32;
  p.chunks = (uint32_t)((n + p.ch - 1) / p.ch);
  p.chunks2 = (p.chunks + kJoin - 1) / kJoin;
  p.blocks = (uint32_t)((n + kSortTile - 1) / kSortTile);
  p.tiles = (uint32_t)((n + kCountTile - 1) / kCountTile);
  p.pdim = (dim + 7) / 8 * 8;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  for (int i = 0; i < 2; ++i) {
    p.key[i] = take(4 * n);
    p.pos[i] = take(4 * n);
  }
  p.hist = take(4ll * 256 * p.blocks);
  p.total = take(4 * 256);
  p.chunk_runs = take(4ll * p.chunks);
  p.tile_runs = take(4ll * p.tiles);
  p.head = take(4 * p.pdim * p.chunks);
  p.tail = take(4 * p.pdim * p.chunks);
  p.head2 = take(4 * p.pdim * p.chunks2);
  p.tail2 = take(4 * p.pdim * p.chunks2);
  p.bytes = at;
  return p;
}

int64_t embed_grad_workspace_bytes(int64_t n, int64_t rows, int32_t dim) {
  (void)rows;
  return embed_grad_plan(n, dim).bytes;
}

template <bool GRAD_F32>
static void launch_segments(const SegKArgs& a, int32_t dout_f32, hipStream_t stream) {
  const unsigned per = 256u >> a.group_shift;
  const unsigned cols = (unsigned)((a.dim + (8 << a.group_shift) - 1) / (8 << a.group_shift));
  const dim3 block(kSegThreads), grid((a.chunks + per - 1) / per, cols), grid2((a.chunks2 + per - 1) / per, cols);
  if (dout_f32)
    hipLaunchKernelGGL((segment_sum_kernel<true, GRAD_F32>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((segment_sum_kernel<false, GRAD_F32>), grid, block, 0, stream, a);
  if (a.chunks > 1) hipLaunchKernelGGL((segment_join_kernel<GRAD_F32>), grid2, block, 0, stream, a);
  if (a.chunks2 > 1) hipLaunchKernelGGL((segment_finish_kernel<GRAD_F32>), grid2, block, 0, stream, a);
}

hipError_t launch_embed_grad(const EmbedGradArgs& g, hipStream_t stream) {
  (void)hipGetLastError();
  const size_t grad_size = g.grad_f32 ? 4 : 2, dout_size = g.dout_f32 ? 4 : 2;
  const int64_t n = g.T * g.cols;
  const int32_t grad_vec = ((uintptr_t)g.grad % 16 == 0 && g.grad_ld * grad_size % 16 == 0) ? 1 : 0;
  if (g.mode == ENGRAM_GRAD_DENSE) {
    const uint32_t chunks = (uint32_t)((g.dim + 7) / 8);
    const int64_t blocks = (g.rows * chunks + 255) / 256;
    const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
    if (g.grad_f32)
      hipLaunchKernelGGL((zero_rows_kernel<true>), grid, dim3(256), 0, stream, g.grad, g.rows, g.dim, g.grad_ld, grad_vec, chunks);
    else
      hipLaunchKernelGGL((zero_rows_kernel<false>), grid, dim3(256), 0, stream, g.grad, g.rows, g.dim, g.grad_ld, grad_vec, chunks);
  }
  char* w = static_cast<char*>(g.work);
  const EmbedGradPlan p = embed_grad_plan(n, g.dim);
  RunKArgs r;
  if (n == 0) {
    if (g.mode == ENGRAM_GRAD_SPARSE) {
      r = RunKArgs{};
      r.count = g.count;
      hipLaunchKernelGGL(run_scan_kernel, dim3(1), dim3(256), 0, stream, r);
    }
    return hipGetLastError();
  }

  SortKArgs s;
  s.ids = g.ids;
  s.ids_ld = g.ids_ld;
  s.n = p.n;
  s.rows = (uint32_t)g.rows;
  s.cols = (uint32_t)g.cols;
  s.blocks = p.blocks;
  s.div_cols = make_fastdiv(s.cols);
  s.hist = reinterpret_cast<uint32_t*>(w + p.hist);
  s.total = reinterpret_cast<uint32_t*>(w + p.total);
  int cur = 0;
  for (uint32_t shift = 0; shift < 32 && (shift == 0 || (s.rows >> shift) != 0); shift += 8) {
    s.shift = shift;
    s.key_in = reinterpret_cast<const uint32_t*>(w + p.key[cur]);
    s.pos_in = reinterpret_cast<const uint32_t*>(w + p.pos[cur]);
    cur ^= 1;
    s.key_out = reinterpret_cast<uint32_t*>(w + p.key[cur]);
    s.pos_out = reinterpret_cast<uint32_t*>(w + p.pos[cur]);
    if (shift == 0) hipLaunchKernelGGL((sort_count_kernel<true>), dim3(p.blocks), dim3(kSortThreads), 0, stream, s);
    else hipLaunchKernelGGL((sort_count_kernel<false>), dim3(p.blocks), dim3(kSortThreads), 0, stream, s);
    hipLaunchKernelGGL(sort_scan_kernel, dim3(256), dim3(256), 0, stream, s);
    if (shift == 0) hipLaunchKernelGGL((sort_scatter_kernel<true>), dim3(p.blocks), dim3(kSortThreads), 0, stream, s);
    else hipLaunchKernelGGL((sort_scatter_kernel<false>), dim3(p.blocks), dim3(kSortThreads), 0, stream, s);
  }
  const uint32_t* key = reinterpret_cast<const uint32_t*>(w + p.key[cur]);
  if (g.mode == ENGRAM_GRAD_SPARSE) {
    r.key = key;
    r.n = p.n;
    r.rows = s.rows;
    r.ch = p.ch;
    r.tiles = p.tiles;
    r.chunk_runs = reinterpret_cast<uint32_t*>(w + p.chunk_runs);
    r.tile_runs = reinterpret_cast<uint32_t*>(w + p.tile_runs);
    r.unique = g.unique;
    r.count = g.count;
    hipLaunchKernelGGL(run_count_kernel, dim3(p.tiles), dim3(256), 0, stream, r);
    hipLaunchKernelGGL(run_scan_kernel, dim3(1), dim3(256), 0, stream, r);
  }
  SegKArgs a;
  a.key = key;
  a.pos = reinterpret_cast<const uint32_t*>(w + p.pos[cur]);
  a.dout = g.dout;
  a.grad = g.grad;
  a.head = reinterpret_cast<float*>(w + p.head);
  a.tail = reinterpret_cast<float*>(w + p.tail);
  a.head2 = reinterpret_cast<float*>(w + p.head2);
  a.tail2 = reinterpret_cast<float*>(w + p.tail2);
  a.chunk_runs = reinterpret_cast<const uint32_t*>(w + p.chunk_runs);
  a.tile_runs = reinterpret_cast<const uint32_t*>(w + p.tile_runs);
  a.unique = g.unique;
  a.dout_ld = g.dout_ld;
  a.seg_pitch = g.seg_pitch;
  a.grad_ld = g.grad_ld;
  a.n = p.n;
  a.rows = s.rows;
  a.cols = s.cols;
  a.ch = p.ch;
  a.chunks = p.chunks;
  a.chunks2 = p.chunks2;
  a.dim = g.dim;
  a.pdim = (int32_t)p.pdim;
  a.mode = g.mode;
  a.scale = g.scale;
  a.dout_vec = ((uintptr_t)g.dout % 16 == 0 && g.dout_ld * dout_size % 16 == 0 && g.seg_pitch * dout_size % 16 == 0 &&
                g.seg_pitch >= p.pdim)
                   ? 1
                   : 0;
  a.grad_vec = grad_vec;
  a.div_cols = s.div_cols;
  a.group_shift = 2;
  while (a.group_shift < 8 && (8 << a.group_shift) < g.dim) ++a.group_shift;
  if (g.grad_f32) launch_segments<true>(a, g.dout_f32, stream);
  else launch_segments<false>(a, g.dout_f32, stream);
  return hipGetLastError();
}

}  // namespace engram
