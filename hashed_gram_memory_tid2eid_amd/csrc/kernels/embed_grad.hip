// embed_grad.hip -- the gradient of the lookup in embed.hip, by sorted tokens.  Included into
// engram_device.hip after embed.hip, whose helpers it uses.
//
//   grad[r][d] = scale * sum over the places (t, c) with ids[t][c] = r of dout[t][c seg_pitch + d]
//
// The places are sorted by row id, stably (id -1 and ids outside the table sort behind every
// row), so a row's places are one run.  Up to kMergeSort places each finds its place in the
// sorted list by counting, in one launch or two; more take a radix sort over as many bits as
// the table's row count has, three launches for each digit of up to 10 bits.  The zeros of a
// dense gradient's other rows are written by workgroups beside those that sum, which find in the sorted list which rows
// those are, so that every row is written once (16,384 tokens, 129,280 x 4,096 fp32: 435 us,
// 5.2 TB/s; cleared whole beside the sort 475).
//
// The sorted list is cut into chunks of `ch` places; a group of lanes owns one chunk and one
// range of columns, 8 per lane (two runs of 4, so that fp32 rows are read and written in
// whole lines), and walks it with fp32 sums in registers.  A run inside a
// chunk is finished there and written once.  Runs that cross chunks leave partial rows:
// `head` (a run that came in from the chunk before) and `tail` (a run that starts here and
// goes on); the group of the chunk where such a run starts adds them up.  So that a row that
// holds much of the batch is not one long chain, units of kUnit chunks inside one run are
// added first, each by a group of its own.  Nothing is added by atomics: the order of every
// sum follows the sorted places, so results repeat bit for bit.

namespace engram {

// (16 waves of 2 places a lane: 393,216 places in 4 waves of 8 took 11 us longer)
constexpr int kSortThreads = 1024, kSortItems = 2, kSortTile = kSortThreads * kSortItems;
constexpr int kSortBits = 10;     // digit of the sort over many workgroups
constexpr int kSmallThreads = 1024;
constexpr int kCountSort = 4096;  // up to this many places are ranked by counting,
constexpr int kMergeTile = 256, kMergeSort = 32768;  // up to this many by tiles
constexpr int kSegThreads = 256;
constexpr int kUnit = 32;         // chunks per unit
constexpr int64_t kChunkLanes = 131072;  // lanes that a longer chunk has to leave: 8 waves on every CU
constexpr int kFewUnits = 16;     // up to this many units, runs add their heads without unit sums
                                  // (up to 32: 3,000 places 2 us less, all of one row 70 us more)
constexpr uint32_t kZeroScan = 2048;  // places that are looked at one by one for rows without one
constexpr int kCountTile = 1024;  // sorted places per workgroup of the run count

struct SortKArgs {
  const int32_t* ids;     // first pass: [T][ids_ld]
  const uint32_t* key_in; // later passes
  const uint32_t* pos_in;
  uint32_t* key_out;
  uint32_t* pos_out;
  uint32_t* hist;         // [blocks][digits]
  uint32_t* total;        // [digits]
  int64_t ids_ld;
  uint32_t n, rows, cols, blocks, shift, bits;
  FastDiv div_cols;
};

// the sort key of place i: its row, or `rows` where it has none
template <bool LATCH>
__device__ __forceinline__ uint32_t place_key(const SortKArgs& a, uint32_t i) {
  const uint32_t t = fdiv(i, a.div_cols);
  const int32_t id = a.ids[(int64_t)t * a.ids_ld + (i - t * a.cols)];
  if (id >= 0 && (uint32_t)id < a.rows) return (uint32_t)id;
  if (LATCH && id != -1) latch_error(ENGRAM_E_ROW_RANGE);
  return a.rows;
}

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortKArgs a) {
  __shared__ uint32_t cnt[1 << kSortBits];
  const uint32_t digits = 1u << a.bits;
  for (uint32_t d = threadIdx.x; d < digits; d += kSortThreads) cnt[d] = 0;
  __syncthreads();
  const uint32_t base = blockIdx.x * kSortTile;
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    const uint32_t at = base + i * kSortThreads + threadIdx.x;
    if (at < a.n) atomicAdd(&cnt[((FIRST ? place_key<true>(a, at) : a.key_in[at]) >> a.shift) & (digits - 1)], 1u);
  }
  __syncthreads();
  for (uint32_t d = threadIdx.x; d < digits; d += kSortThreads) a.hist[(int64_t)blockIdx.x * digits + d] = cnt[d];
}

__device__ __forceinline__ uint32_t wave_inclusive(uint32_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)v, off, 64);
    if (lane >= off) v += o;
  }
  return v;
}

// exclusive sum over the workgroup's threads; *all receives the total
template <int THREADS>
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* wsum, uint32_t* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t s = wave_inclusive(v);
  __syncthreads();  // the last call's readers are done with wsum
  if (lane == 63) wsum[wave] = s;
  __syncthreads();
  uint32_t before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    if (w < wave) before += wsum[w];
    sum += wsum[w];
  }
  *all = sum;
  return before + s - v;
}

// A lane per digit: its counts over the blocks become exclusive sums.  Each wave adds up a part
// of the blocks, then writes its sums behind those of the waves before it.
__global__ __launch_bounds__(kSortThreads) void sort_scan_kernel(SortKArgs a) {
  constexpr uint32_t WAVES = kSortThreads / 64;
  __shared__ uint32_t part[WAVES][64];
  const uint32_t digits = 1u << a.bits, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, digit = blockIdx.x * 64 + lane;
  const uint32_t per = (a.blocks + WAVES - 1) / WAVES, b0 = min(a.blocks, wave * per), b1 = min(a.blocks, b0 + per);
  uint32_t* h = a.hist + min(digit, digits - 1);
  uint32_t sum = 0;
#pragma unroll 8
  for (uint32_t b = b0; b < b1; ++b) sum += h[(int64_t)b * digits];
  part[wave][lane] = sum;
  __syncthreads();
  if (digit >= digits) return;
  uint32_t carry = 0;
  for (uint32_t w = 0; w < wave; ++w) carry += part[w][lane];
  if (wave == WAVES - 1) a.total[digit] = carry + sum;
#pragma unroll 8
  for (uint32_t b = b0; b < b1; ++b) {
    const uint32_t v = h[(int64_t)b * digits];
    h[(int64_t)b * digits] = carry;
    carry += v;
  }
}

// Stable rank of a wave's 64 keys among those with the same digit: the lanes with one digit
// find each other by a ballot per bit, and the first of them moves the wave's count of the
// digit on.
template <typename COUNT>
__device__ __forceinline__ uint32_t wave_rank(uint32_t d, int bits, bool live, COUNT* count) {
  uint64_t peers = __ballot(live);
  for (int b = 0; b < bits; ++b) {  // uniform
    const bool bit = (d >> b) & 1u;
    const uint64_t m = __ballot(bit);
    peers &= bit ? m : ~m;
  }
  const uint32_t below = (uint32_t)__popcll(peers & ((1ull << (threadIdx.x & 63)) - 1ull));
  const uint32_t before = *count;
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");  // every lane has read before one writes: LDS keeps a wave's order
  if (live && below == 0) *count = (COUNT)(before + (uint32_t)__popcll(peers));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
  return before + below;
}

// Stable scatter of one pass: wave w owns places [64 kSortItems w, + 64 kSortItems) of the tile
template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(SortKArgs a) {
  constexpr int PER = (1 << kSortBits) / kSortThreads;  // digits per thread
  constexpr int WAVES = kSortThreads / 64;
  __shared__ uint32_t cnt[WAVES][1 << kSortBits];
  __shared__ uint32_t wsum[WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t digits = 1u << a.bits;
  uint32_t key[kSortItems], pos[kSortItems], rank[kSortItems];
  const uint32_t base = blockIdx.x * kSortTile + wave * (64 * kSortItems);
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    const uint32_t at = base + i * 64 + lane;
    key[i] = at >= a.n ? 0u : FIRST ? place_key<false>(a, at) : a.key_in[at];
    pos[i] = at >= a.n ? 0u : FIRST ? at : a.pos_in[at];
  }
  uint32_t first[PER], sum = 0;  // thread's digits PER tid ..: first output place of this block
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const uint32_t d = tid * PER + e;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) cnt[w][d] = 0;
    first[e] = sum + (d < digits ? a.hist[(int64_t)blockIdx.x * digits + d] : 0u);
    sum += d < digits ? a.total[d] : 0u;
  }
  uint32_t all;
  const uint32_t before = block_exclusive<kSortThreads>(sum, wsum, &all);  // its barriers publish cnt
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    const uint32_t d = (key[i] >> a.shift) & (digits - 1);
    rank[i] = wave_rank(d, (int)a.bits, base + i * 64 + lane < a.n, &cnt[wave][d]);
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    uint32_t run = before + first[e];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const uint32_t c = cnt[w][tid * PER + e];
      cnt[w][tid * PER + e] = run;
      run += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    if (base + i * 64 + lane >= a.n) continue;
    const uint32_t to = cnt[wave][(key[i] >> a.shift) & (digits - 1)] + rank[i];
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
  int32_t* unique;       // null: no names wanted
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
  const uint32_t ex = block_exclusive<256>(c, wsum, &all);
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
    const uint32_t ex = block_exclusive<256>(v, wsum, &all);
    if (at < a.tiles) a.tile_runs[at] = carry + ex;
    carry += all;
  }
  if (threadIdx.x == 0) *a.count = (int32_t)carry;
}

// ---- a short list: sorted by one workgroup, in LDS -------------------------------------

// Rank of a place = the places with a smaller key, and those before it with the same.  Each
// workgroup holds all keys in LDS and ranks 64 / SPLIT places: SPLIT lanes of every wave count
// for one place over equal shares of the list, a compare and an add with carry a pair.  The
// whole gradient of 12,288 rows of 128 with this or with a sort by digits in one workgroup: 1
// place 8 us against 15, 3,000 places 17 against 25.
template <int SPLIT>
__global__ __launch_bounds__(kSmallThreads) void sort_count_all_kernel(SortKArgs a) {
  constexpr uint32_t PLACES = 64 / SPLIT, SHARES = kSmallThreads / PLACES;
  __shared__ __attribute__((aligned(16))) uint32_t keys[kCountSort];
  // (one address a wave where the shares are the waves')
  const uint32_t tid = threadIdx.x, lane = tid % PLACES;
  const uint32_t part = SPLIT == 1 ? (uint32_t)__builtin_amdgcn_readfirstlane(tid / PLACES) : tid / PLACES;
  const uint32_t share = (a.n + SHARES * 8 - 1) / (SHARES * 8) * 8;  // places per share, 8 at a time
  for (uint32_t i = tid; i < share * SHARES; i += kSmallThreads)
    keys[i] = i >= a.n ? 0xFFFFFFFFu : blockIdx.x == 0 ? place_key<true>(a, i) : place_key<false>(a, i);
  __syncthreads();
  const uint32_t p0 = blockIdx.x * PLACES, me = p0 + lane;
  const uint32_t key = keys[min(me, a.n - 1)];
  const uint32_t j0 = part * share, j1 = j0 + share;
  // before the workgroup's places an equal key counts, behind them it does not
  uint32_t below = 0;
  auto count = [&](uint32_t from, uint32_t to, uint32_t limit) {
    for (uint32_t j = from; j < to; j += 8) {
      uint32_t k[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] = keys[j + e];
#pragma unroll
      for (int e = 0; e < 8; ++e) below += k[e] < limit ? 1u : 0u;
    }
  };
  const uint32_t m0 = min(max(j0, p0), j1), m1 = min(max(j0, p0 + PLACES), j1);
  count(j0, m0, key + 1);
  for (uint32_t j = m0; j < m1; ++j) below += keys[j] < key + (j < me ? 1u : 0u) ? 1u : 0u;
  count(m1, j1, key);
  __syncthreads();  // the keys are done with
  keys[tid] = below;
  __syncthreads();
  if (tid >= PLACES || me >= a.n) return;
  uint32_t rank = 0;
#pragma unroll 16
  for (uint32_t w = 0; w < SHARES; ++w) rank += keys[w * PLACES + lane];
  a.key_out[rank] = key;
  a.pos_out[rank] = me;
}

template <int SPLIT>
static void launch_count_all(const SortKArgs& s, hipStream_t stream) {
  const unsigned grid = (s.n * SPLIT + 63) / 64;
  if (grid > 0) hipLaunchKernelGGL((sort_count_all_kernel<SPLIT>), dim3(grid), dim3(kSmallThreads), 0, stream, s);
}

// Longer lists: each workgroup sorts a tile by counting, then every place is looked up in every
// tile.  A workgroup holds all tiles in LDS and ranks 64 places of one tile, a lane each; its
// waves take the tiles in turn.  16,384 places: 5 + 5 us; all pairs counted 29 us, which is the time
// to read the keys from LDS once per workgroup.
__global__ __launch_bounds__(kSmallThreads) void sort_tile_kernel(SortKArgs a) {
  constexpr uint32_t SHARES = kSmallThreads / kMergeTile, SHARE = kMergeTile / SHARES;  // waves per place; places a wave looks at
  static_assert(SHARE == 64, "a wave's places are one share");
  __shared__ __attribute__((aligned(16))) uint32_t keys[kMergeTile];
  __shared__ uint32_t counts[SHARES][kMergeTile];
  const uint32_t tid = threadIdx.x, p = tid % kMergeTile, at = blockIdx.x * kMergeTile + p;
  const uint32_t mine = (uint32_t)__builtin_amdgcn_readfirstlane(p / SHARE);
  const uint32_t share = (uint32_t)__builtin_amdgcn_readfirstlane(tid / kMergeTile);
  if (tid < kMergeTile) keys[tid] = at < a.n ? place_key<true>(a, at) : 0xFFFFFFFFu;
  __syncthreads();
  const uint32_t key = keys[p], *from = keys + share * SHARE;
  uint32_t below = 0;
  if (share == mine) {
#pragma unroll 16
    for (uint32_t j = 0; j < SHARE; ++j) below += from[j] < key + (j < p % SHARE ? 1u : 0u) ? 1u : 0u;
  } else {
    const uint32_t limit = key + (share < mine ? 1u : 0u);
#pragma unroll 16
    for (uint32_t j = 0; j < SHARE; ++j) below += from[j] < limit ? 1u : 0u;
  }
  counts[share][p] = below;
  __syncthreads();
  if (tid >= kMergeTile || at >= a.n) return;
  uint32_t rank = blockIdx.x * kMergeTile;
#pragma unroll
  for (uint32_t e = 0; e < SHARES; ++e) rank += counts[e][p];
  a.key_out[rank] = key;
  a.pos_out[rank] = at;
}

__global__ __launch_bounds__(kSmallThreads) void sort_merge_kernel(SortKArgs a) {
  constexpr uint32_t WAVES = kSmallThreads / 64;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem);  // whole tiles
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = (uint32_t)__builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t tiles = (a.n + kMergeTile - 1) / kMergeTile;
  for (uint32_t i = tid * 4; i < tiles * kMergeTile; i += kSmallThreads * 4) {
    u32x4 k;
    if (i + 4 <= a.n) {
      k = *reinterpret_cast<const u32x4*>(a.key_in + i);
    } else {
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) k[e] = i + e < a.n ? a.key_in[i + e] : 0xFFFFFFFFu;
    }
    *reinterpret_cast<u32x4*>(keys + i) = k;
  }
  __syncthreads();
  const uint32_t p0 = blockIdx.x * 64, me = p0 + lane, own = p0 / kMergeTile;
  const uint32_t key = keys[me];
  uint32_t below = 0;
#pragma unroll 4
  for (uint32_t t = wave; t < tiles; t += WAVES) {
    // an equal key of an earlier tile counts, of a later one it does not
    const uint32_t limit = key + (t < own ? 1u : 0u);
    const uint32_t* tile = keys + t * kMergeTile;
    uint32_t c = 0;
#pragma unroll
    for (uint32_t step = kMergeTile / 2; step > 0; step /= 2) c += tile[c + step - 1] < limit ? step : 0u;
    c += tile[c] < limit ? 1u : 0u;
    below += t == own ? me % kMergeTile : c;
  }
  __syncthreads();  // the keys are done with
  keys[tid] = below;
  __syncthreads();
  if (wave != 0 || me >= a.n) return;
  uint32_t rank = 0;
#pragma unroll
  for (uint32_t w = 0; w < WAVES; ++w) rank += keys[w * 64 + lane];
  a.key_out[rank] = key;
  a.pos_out[rank] = a.pos_in[me];
}

// the runs of a list of up to kCountSort places, in one workgroup
__global__ __launch_bounds__(kSmallThreads) void run_small_kernel(RunKArgs r) {
  constexpr uint32_t PER = kCountSort / kSmallThreads;
  __shared__ uint32_t wsum[kSmallThreads / 64];
  const uint32_t tid = threadIdx.x, s0 = tid * PER;
  uint32_t c = 0, last = s0 > 0 && s0 < r.n ? r.key[s0 - 1] : r.rows;
#pragma unroll
  for (uint32_t e = 0; e < PER; ++e) {
    if (s0 + e >= r.n) continue;
    const uint32_t k = r.key[s0 + e];
    c += k < r.rows && k != last ? 1u : 0u;
    last = k;
    r.unique[s0 + e] = -1;
  }
  uint32_t all;
  const uint32_t before = block_exclusive<kSmallThreads>(c, wsum, &all);
  if (s0 < r.n && s0 % r.ch == 0) r.chunk_runs[s0 / r.ch] = before;  // chunks are multiples of PER places
  if (tid < r.tiles) r.tile_runs[tid] = 0;  // chunk_runs count from the start of the list
  if (tid == 0) *r.count = (int32_t)all;
}

// ---- sums over the runs ------------------------------------------------------------

struct SegKArgs {
  const uint32_t* key;
  const uint32_t* pos;
  const void* dout;
  void* grad;
  float* head;    // [chunks][pdim]
  float* tail;
  float* unit;    // [units][pdim]: sums of units inside one run
  const uint32_t* chunk_runs;
  const uint32_t* tile_runs;
  int32_t* unique;
  int64_t dout_ld, seg_pitch, grad_ld;
  uint32_t n, rows, cols, ch, chunks, units;
  int32_t dim, pdim, mode;
  float scale;
  int32_t dout_vec, grad_vec;
  uint32_t group_shift;  // log2 of the lanes per group
  uint32_t blocks;       // workgroups that sum, per range of columns
  uint32_t sum_blocks;   // over all ranges; those behind them write zeros (dense)
  FastDiv div_cols;
  uint32_t zero_rows;    // rows per workgroup that writes zeros, at most kSegThreads
  uint32_t row_units;    // a row in units of 16 bytes, or of its elements where rows are not aligned
  FastDiv div_units;
};

struct SegPlace {
  uint32_t unit;  // the chunk (or unit) this group owns
  int32_t col;    // the lane's first 4 columns; its other 4 are `other` columns on
  int32_t other;
};

// workgroup `block` of `blocks` per range of columns
__device__ __forceinline__ SegPlace seg_place(const SegKArgs& a, uint32_t block, uint32_t blocks) {
  const uint32_t lane = threadIdx.x & ((1u << a.group_shift) - 1u);
  const uint32_t range = block / blocks;
  SegPlace p;
  p.unit = ((block - range * blocks) << (8 - a.group_shift)) + (threadIdx.x >> a.group_shift);
  p.other = 4 << a.group_shift;
  p.col = (int32_t)(range * 2 * p.other + lane * 4);
  return p;
}

// zeros for the rows of a dense gradient that no place names: rows zero_rows * block .. of them
template <bool GRAD_F32>
__device__ __forceinline__ void zero_other_rows(const SegKArgs& a, uint32_t block) {
  __shared__ uint8_t named[kSegThreads];
  __shared__ uint32_t below[2];
  const uint32_t r0 = block * a.zero_rows, count = min(a.zero_rows, a.rows - r0), tid = threadIdx.x;
  named[tid] = 0;
  if (tid < 2) below[tid] = 0;
  __syncthreads();
  // the last place of every 256th part of the list says where the rows' places lie (one load
  // where a search takes one a step: 3,000 places, 12,288 x 128 fp32 17 us against 19)
  const uint32_t step = (a.n + kSegThreads - 1) / kSegThreads;
  const uint32_t probe = a.n > 0 ? a.key[min((tid + 1) * step, a.n) - 1] : 0u;
  const uint64_t low = __ballot(probe < r0), high = __ballot(probe < r0 + count);
  if ((tid & 63) == 0) {
    atomicAdd(&below[0], (uint32_t)__popcll(low));
    atomicAdd(&below[1], (uint32_t)__popcll(high));
  }
  __syncthreads();
  const uint32_t from = min(below[0] * step, a.n), to = min((below[1] + 1) * step, a.n);
  if (to - from <= kZeroScan) {
#pragma unroll
    for (uint32_t e = 0; e < kZeroScan; e += kSegThreads) {
      const uint32_t i = from + e + tid;
      const uint32_t r = i < to ? a.key[i] - r0 : count;
      if (r < count) named[r] = 1;
    }
  } else if (tid < count) {
    uint32_t lo = from, hi = to;  // the first place at or behind the row
    while (lo < hi) {
      const uint32_t mid = (lo + hi) / 2;
      if (a.key[mid] < r0 + tid) lo = mid + 1;
      else hi = mid;
    }
    named[tid] = lo < a.n && a.key[lo] == r0 + tid ? 1 : 0;
  }
  __syncthreads();
  constexpr int SIZE = GRAD_F32 ? 4 : 2;
  char* base = static_cast<char*>(a.grad) + (int64_t)r0 * a.grad_ld * SIZE;
  const u32x4 zero = {};
  for (uint32_t i = tid; i < count * a.row_units; i += kSegThreads) {
    const uint32_t r = fdiv(i, a.div_units), unit = i - r * a.row_units;
    if (named[r]) continue;
    char* at = base + (int64_t)r * a.grad_ld * SIZE;
    if (a.grad_vec) __builtin_nontemporal_store(zero, reinterpret_cast<u32x4*>(at) + unit);
    else if (GRAD_F32) reinterpret_cast<float*>(at)[unit] = 0.0f;
    else reinterpret_cast<unsigned short*>(at)[unit] = 0;
  }
}

// runs that start before sorted place i, the first of its chunk
__device__ __forceinline__ uint32_t runs_before(const SegKArgs& a, uint32_t i) {
  return a.tile_runs[i / kCountTile] + a.chunk_runs[i / a.ch];
}

template <bool GRAD_F32>
__device__ __forceinline__ void write_row(const SegKArgs& a, uint32_t key, uint32_t run, const SegPlace& p, const float* acc) {
  const bool sparse = a.mode == ENGRAM_GRAD_SPARSE;
  const int64_t row = (int64_t)(sparse ? run : key) * a.grad_ld;
  if (sparse && p.col == 0) a.unique[run] = (int32_t)key;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int32_t col = p.col + h * p.other;
    const int n = min(4, a.dim - col);
    if (n <= 0) continue;
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = acc[4 * h + i] * a.scale;
    if (a.mode == ENGRAM_GRAD_ACCUMULATE) {
      float old[4];
      load_chunk<GRAD_F32, 4>(a.grad, row + col, n, a.grad_vec != 0, old);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] += old[i];
    }
    // past the caches, which keep dout's rows: 16,384 x 24 places of 256 171 us against 198
    store_chunk<GRAD_F32, 4, true>(a.grad, row + col, n, a.grad_vec != 0, f);
  }
}

// partial rows are padded to whole lanes' columns
__device__ __forceinline__ void put_partial(float* to, const SegKArgs& a, const SegPlace& p, const float* acc) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    *reinterpret_cast<f32x4*>(to + (int64_t)p.unit * a.pdim + p.col + h * p.other) =
        f32x4{acc[4 * h], acc[4 * h + 1], acc[4 * h + 2], acc[4 * h + 3]};
}

// acc += rows u0 .. u1 - 1 of a partial array, in order, many in flight
__device__ __forceinline__ void add_partials(const float* from, const SegKArgs& a, uint32_t u0, uint32_t u1,
                                             const SegPlace& p, float* acc) {
  constexpr int U = 8;
  for (uint32_t u = u0; u < u1; u += U) {
    f32x4 v[U][2];
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const float* src = from + (int64_t)min(u + e, u1 - 1) * a.pdim + p.col;
      v[e][0] = *reinterpret_cast<const f32x4*>(src);
      v[e][1] = *reinterpret_cast<const f32x4*>(src + p.other);
    }
#pragma unroll
    for (int e = 0; e < U; ++e)
      if (u + e < u1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[i] += v[e][0][i];
          acc[4 + i] += v[e][1][i];
        }
      }
  }
}

__device__ __forceinline__ void clear8(float* acc) {
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
}

// a lane's 8 columns of a row as they are loaded, and as floats
template <bool F32>
struct RawChunk {
  uint32_t w[F32 ? 8 : 4];
  // vec: segments start on 16 bytes and hold the columns up to the next multiple of 4
  __device__ __forceinline__ void load(const void* base, int64_t row, const SegPlace& p, int32_t dim, bool vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int32_t col = p.col + h * p.other;
      const int64_t at = row + col;
      if (col >= dim) {
#pragma unroll
        for (int i = 0; i < (F32 ? 4 : 2); ++i) w[(F32 ? 4 : 2) * h + i] = 0u;
      } else if (vec) {
        if (F32) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const float*>(base) + at);
#pragma unroll
          for (int i = 0; i < 4; ++i) w[F32 ? 4 * h + i : 0] = v[i];
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const unsigned short*>(base) + at);
          w[2 * h] = v.x;
          w[2 * h + 1] = v.y;
        }
      } else {
        float f[4];
        load_chunk<F32, 4>(base, at, dim - col, false, f);
        if (F32) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[F32 ? 4 * h + i : 0] = __float_as_uint(f[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) w[2 * h + i] = (__float_as_uint(f[2 * i]) >> 16) | __float_as_uint(f[2 * i + 1]);
        }
      }
    }
  }
  __device__ __forceinline__ void to_float(float* f) const {
    if (F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[F32 ? i : 0]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
};

template <bool DOUT_F32, bool GRAD_F32>
__global__ __launch_bounds__(kSegThreads) void segment_sum_kernel(SegKArgs a) {
  constexpr int U = 4;  // rows in flight per lane (8: fewer waves fit, 70 us against 55 at 16,384 x 24)
  if (blockIdx.x >= a.sum_blocks) {
    zero_other_rows<GRAD_F32>(a, blockIdx.x - a.sum_blocks);
    return;
  }
  const SegPlace p = seg_place(a, blockIdx.x, a.blocks);
  if (p.unit >= a.chunks || p.col >= a.dim) return;
  const uint32_t i0 = p.unit * a.ch, i1 = min(a.n, i0 + a.ch);
  // (a.ch is a multiple of U) the next U places' keys and positions are fetched while the
  // rows of the current ones are on their way
  uint32_t nk[U], np[U];
  auto fetch = [&](uint32_t i) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t at = min(i + u, a.n - 1);
      nk[u] = a.key[at];
      np[u] = a.pos[at];
    }
  };
  const uint32_t left = a.key[max(i0, 1u) - 1], right = a.key[min(i1, a.n - 1)];
  fetch(i0);
  uint32_t cur = nk[0];
  if (cur >= a.rows) return;
  bool started = i0 == 0 || left != cur;
  uint32_t run = 0;
  if (a.mode == ENGRAM_GRAD_SPARSE) run = runs_before(a, i0) - (started ? 0u : 1u);
  float acc[8];
  clear8(acc);
  for (uint32_t i = i0; i < i1; i += U) {
    uint32_t k[U];
    RawChunk<DOUT_F32> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      k[u] = i + u < i1 ? nk[u] : a.rows;
      const uint32_t t = fdiv(np[u], a.div_cols);
      const int64_t row = (int64_t)t * a.dout_ld + (int64_t)(np[u] - t * a.cols) * a.seg_pitch;
      if (k[u] < a.rows) raw[u].load(a.dout, row, p, a.dim, a.dout_vec != 0);
    }
    if (i + U < i1) fetch(i + U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= i1) continue;
      if (k[u] != cur) {
        if (started) write_row<GRAD_F32>(a, cur, run, p, acc);
        else put_partial(a.head, a, p, acc);
        if (k[u] >= a.rows) return;  // the rest has no row
        clear8(acc);
        started = true;
        cur = k[u];
        ++run;
      }
      float f[8];
      raw[u].to_float(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += f[e];
    }
  }
  const bool goes_on = i1 < a.n && right == cur;
  if (!started) put_partial(a.head, a, p, acc);
  else if (goes_on) put_partial(a.tail, a, p, acc);
  else write_row<GRAD_F32>(a, cur, run, p, acc);
}

// sums of the units (kUnit chunks) that a run comes into and leaves: all of it is head rows
__global__ __launch_bounds__(kSegThreads) void segment_unit_kernel(SegKArgs a, uint32_t blocks) {
  const SegPlace p = seg_place(a, blockIdx.x, blocks);
  if (p.unit == 0 || p.unit >= a.units || p.col >= a.dim) return;
  const uint32_t c0 = p.unit * kUnit, c1 = c0 + kUnit;
  const uint32_t k = a.key[c0 * a.ch];
  if (k >= a.rows || a.key[c0 * a.ch - 1] != k || c1 >= a.chunks || a.key[c1 * a.ch] != k)
    return;
  float acc[8];
  clear8(acc);
  add_partials(a.head, a, c0, c1, p, acc);
  put_partial(a.unit, a, p, acc);
}

// the chunk in which a run starts that leaves it adds what the following chunks hold
template <bool GRAD_F32>
__global__ __launch_bounds__(kSegThreads) void segment_finish_kernel(SegKArgs a) {
  const SegPlace p = seg_place(a, blockIdx.x, a.blocks);
  const uint32_t c = p.unit;
  if (c + 1 >= a.chunks) return;  // lanes past the row's columns stay: they look for the end, too
  const uint32_t end = (c + 1) * a.ch;
  const uint32_t k = a.key[end], inside = a.key[end - 1], before = a.key[max(c * a.ch, 1u) - 1];
  if (k >= a.rows || inside != k) return;  // nothing leaves (the same for the whole group)
  if (c > 0 && before == k) return;        // it started earlier
  // `stop`, the first chunk that the run does not come into: the lanes of the group (of the
  // wave, where the group is larger) each look at the last chunk of a block of `step`; while
  // the run covers all blocks they grow, then the block that it ends in is divided
  const uint32_t shift = min(6u, a.group_shift), width = 1u << shift, lane = threadIdx.x & 63;
  const uint32_t me = lane & (width - 1), lowest = lane & ~(width - 1);
  uint32_t stop = c + 2, step = 0;  // step: log2
  for (;;) {
    const uint64_t at = (uint64_t)stop + ((uint64_t)(me + 1) << step) - 1;
    const bool covered = at < a.chunks && a.key[(uint32_t)at * a.ch] == k;
    const uint64_t ended = (__ballot(!covered) >> lowest) & (width == 64 ? ~0ull : (1ull << width) - 1ull);
    const uint32_t blocks = ended != 0 ? (uint32_t)__ffsll((unsigned long long)ended) - 1 : width;
    stop += blocks << step;
    if (ended == 0) step += shift;
    else if (step == 0) break;
    else step -= shift;
  }
  float acc[8];
  clear8(acc);
  add_partials(a.tail, a, c, c + 1, p, acc);
  // heads up to a unit, whole units (the run goes on behind them), heads of the rest
  const uint32_t u0 = (c + kUnit) / kUnit, u1 = (stop - 1) / kUnit;
  if (a.units > kFewUnits && u0 < u1) {
    add_partials(a.head, a, c + 1, u0 * kUnit, p, acc);
    add_partials(a.unit, a, u0, u1, p, acc);
    add_partials(a.head, a, u1 * kUnit, stop, p, acc);
  } else {
    add_partials(a.head, a, c + 1, stop, p, acc);
  }
  const uint32_t run = a.mode == ENGRAM_GRAD_SPARSE ? runs_before(a, end) - 1u : 0u;
  write_row<GRAD_F32>(a, k, run, p, acc);
}

// ---- the workspace and the launches -------------------------------------------------

struct EmbedGradPlan {
  uint32_t n, ch, chunks, units, blocks, tiles, shift;
  int64_t pdim;
  int64_t key[2], pos[2], hist, total, chunk_runs, tile_runs, head, tail, unit, bytes;
};

static EmbedGradPlan embed_grad_plan(int64_t n, int32_t dim) {
  EmbedGradPlan p;
  p.n = (uint32_t)n;
  // partial rows hold whole groups' columns
  p.shift = 2;
  while (p.shift < 8 && (8 << p.shift) < dim) ++p.shift;
  const int64_t group = 8 << p.shift;
  p.pdim = ((int64_t)dim + group - 1) / group * group;
  // places per chunk: as many as leave enough lanes (each walks one chunk's 8 columns) for 8
  // waves on every CU; more places make fewer partial rows.  At least the places in flight of
  // a lane (3,000 places of 128 added to their rows: 16.5 us, in chunks of 8 17.9)
  const int64_t lanes = n * (p.pdim / 8);
  p.ch = lanes / 32 >= kChunkLanes ? 32 : lanes / 16 >= kChunkLanes ? 16 : lanes / 8 >= kChunkLanes ? 8 : 4;
  p.chunks = (uint32_t)((n + p.ch - 1) / p.ch);
  p.units = (p.chunks + kUnit - 1) / kUnit;
  p.blocks = (uint32_t)((n + kSortTile - 1) / kSortTile);
  p.tiles = (uint32_t)((n + kCountTile - 1) / kCountTile);
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
  p.hist = take(4ll * (1 << kSortBits) * p.blocks);
  p.total = take(4 << kSortBits);
  p.chunk_runs = take(4ll * p.chunks);
  p.tile_runs = take(4ll * p.tiles);
  p.head = take(4 * p.pdim * p.chunks);
  p.tail = take(4 * p.pdim * p.chunks);
  p.unit = take(4 * p.pdim * p.units);
  p.bytes = at;
  return p;
}

// What a gradient of up to n places needs at most.  Each longer chunk halves the partial rows,
// so the last list with the shorter chunk may need more than n places do (dim 256: 32,767
// places 17.7 MB, 32,768 9.1 MB); between these steps the need only grows.
int64_t embed_grad_workspace_bytes(int64_t n, int64_t rows, int32_t dim) {
  (void)rows;
  const EmbedGradPlan all = embed_grad_plan(n, dim);
  int64_t most = all.bytes;
  for (int64_t ch = 8; ch <= 32; ch *= 2) {
    const int64_t last = (ch * kChunkLanes - 1) / (all.pdim / 8);  // the last list whose chunks are shorter
    if (last < n) most = std::max(most, embed_grad_plan(last, dim).bytes);
  }
  return most;
}

template <bool GRAD_F32>
static hipError_t launch_segments(SegKArgs& a, int32_t dout_f32, hipStream_t stream) {
  const unsigned per = 256u >> a.group_shift;
  const unsigned cols = (unsigned)((a.dim + (8 << a.group_shift) - 1) / (8 << a.group_shift));
  a.blocks = (a.chunks + per - 1) / per;
  int64_t zeros = 0;  // workgroups that write zeros
  if (a.mode == ENGRAM_GRAD_DENSE) {
    const int64_t row_bytes = (int64_t)a.dim * (GRAD_F32 ? 4 : 2);
    const bool whole = a.grad_vec != 0 && row_bytes % 16 == 0;
    a.grad_vec = whole ? a.grad_vec : 0;
    a.row_units = (uint32_t)(whole ? row_bytes / 16 : a.dim);
    a.div_units = make_fastdiv(a.row_units);
    // some 256 KB each, which hides the search; less where that gives fewer than four to a CU
    // (1,195 places into 2,412 rows of 538, which no vector store fits, 40 us -> 13 us)
    const int64_t rows = std::min((int64_t)(256 << 10) / row_bytes, (int64_t)a.rows / 1024);
    a.zero_rows = (uint32_t)(rows < 1 ? 1 : rows > kSegThreads ? kSegThreads : rows);
    zeros = ((int64_t)a.rows + a.zero_rows - 1) / a.zero_rows;
  }
  const int64_t sums = (int64_t)a.blocks * cols;
  if (sums + zeros > 0x7FFFFFFF) return hipErrorInvalidValue;
  a.sum_blocks = (uint32_t)sums;
  const dim3 block(kSegThreads), grid((unsigned)(sums + zeros));
  if (grid.x > 0) {
    if (dout_f32)
      hipLaunchKernelGGL((segment_sum_kernel<true, GRAD_F32>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((segment_sum_kernel<false, GRAD_F32>), grid, block, 0, stream, a);
  }
  if (a.units > kFewUnits) {
    const unsigned blocks = (a.units + per - 1) / per;
    hipLaunchKernelGGL(segment_unit_kernel, dim3(blocks * cols), block, 0, stream, a, blocks);
  }
  if (a.chunks > 1) hipLaunchKernelGGL((segment_finish_kernel<GRAD_F32>), dim3((unsigned)sums), block, 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_embed_grad(const EmbedGradArgs& g, hipStream_t stream) {
  (void)hipGetLastError();
  const size_t grad_size = g.grad_f32 ? 4 : 2, dout_size = g.dout_f32 ? 4 : 2;
  const int64_t n = g.T * g.cols;
  const bool sparse = g.mode == ENGRAM_GRAD_SPARSE;
  const int32_t grad_vec = ((uintptr_t)g.grad % 16 == 0 && g.grad_ld * grad_size % 16 == 0) ? 1 : 0;
  const bool small = n <= kMergeSort;
  char* w = static_cast<char*>(g.work);
  RunKArgs r = {};
  if (n == 0 && sparse) {
    r.count = g.count;
    hipLaunchKernelGGL(run_scan_kernel, dim3(1), dim3(256), 0, stream, r);
    return hipGetLastError();
  }
  const EmbedGradPlan p = embed_grad_plan(n, g.dim);

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
  r.n = p.n;
  r.rows = s.rows;
  r.ch = p.ch;
  r.tiles = p.tiles;
  r.chunk_runs = reinterpret_cast<uint32_t*>(w + p.chunk_runs);
  r.tile_runs = reinterpret_cast<uint32_t*>(w + p.tile_runs);
  r.unique = sparse ? g.unique : nullptr;
  r.count = g.count;
  // digits: the key's bits (keys go up to `rows`) in as few passes as the widest digit allows
  uint32_t bits = 1;
  while (bits < 32 && (s.rows >> bits) != 0) ++bits;
  const uint32_t passes = (bits + kSortBits - 1) / kSortBits;
  s.bits = (bits + passes - 1) / passes;
  int cur = 0;
  if (small) {
    s.shift = 0;
    s.key_in = s.pos_in = nullptr;
    s.key_out = reinterpret_cast<uint32_t*>(w + p.key[0]);
    s.pos_out = reinterpret_cast<uint32_t*>(w + p.pos[0]);
    if (n > kCountSort) {
      const unsigned tiles = (p.n + kMergeTile - 1) / kMergeTile;
      static std::atomic<uint64_t> lds_set{0};
      const hipError_t e =
          ensure_dynamic_lds(reinterpret_cast<const void*>(&sort_merge_kernel), kMergeSort * 4, lds_set);
      if (e != hipSuccess) return e;
      hipLaunchKernelGGL(sort_tile_kernel, dim3(tiles), dim3(kSmallThreads), 0, stream, s);
      s.key_in = s.key_out;
      s.pos_in = s.pos_out;
      cur = 1;
      s.key_out = reinterpret_cast<uint32_t*>(w + p.key[1]);
      s.pos_out = reinterpret_cast<uint32_t*>(w + p.pos[1]);
      hipLaunchKernelGGL(sort_merge_kernel, dim3((p.n + 63) / 64), dim3(kSmallThreads), tiles * kMergeTile * 4, stream, s);
    } else if (n > 1024) {  // the counts take less time than their sum in a shorter list
      launch_count_all<4>(s, stream);
    } else {
      launch_count_all<1>(s, stream);
    }
  } else {
    for (uint32_t pass = 0; pass < passes; ++pass) {
      s.shift = pass * s.bits;
      s.key_in = reinterpret_cast<const uint32_t*>(w + p.key[cur]);
      s.pos_in = reinterpret_cast<const uint32_t*>(w + p.pos[cur]);
      cur ^= 1;
      s.key_out = reinterpret_cast<uint32_t*>(w + p.key[cur]);
      s.pos_out = reinterpret_cast<uint32_t*>(w + p.pos[cur]);
      const dim3 grid(p.blocks), block(kSortThreads);
      if (pass == 0) hipLaunchKernelGGL((sort_count_kernel<true>), grid, block, 0, stream, s);
      else hipLaunchKernelGGL((sort_count_kernel<false>), grid, block, 0, stream, s);
      hipLaunchKernelGGL(sort_scan_kernel, dim3(((1u << s.bits) + 63) / 64), block, 0, stream, s);
      if (pass == 0) hipLaunchKernelGGL((sort_scatter_kernel<true>), grid, block, 0, stream, s);
      else hipLaunchKernelGGL((sort_scatter_kernel<false>), grid, block, 0, stream, s);
    }
  }
  r.key = reinterpret_cast<const uint32_t*>(w + p.key[cur]);
  if (sparse && n <= kCountSort) {
    hipLaunchKernelGGL(run_small_kernel, dim3(1), dim3(kSmallThreads), 0, stream, r);
  } else if (sparse) {
    hipLaunchKernelGGL(run_count_kernel, dim3(p.tiles), dim3(256), 0, stream, r);
    hipLaunchKernelGGL(run_scan_kernel, dim3(1), dim3(256), 0, stream, r);
  }
  SegKArgs a;
  a.key = reinterpret_cast<const uint32_t*>(w + p.key[cur]);
  a.pos = reinterpret_cast<const uint32_t*>(w + p.pos[cur]);
  a.dout = g.dout;
  a.grad = g.grad;
  a.head = reinterpret_cast<float*>(w + p.head);
  a.tail = reinterpret_cast<float*>(w + p.tail);
  a.unit = reinterpret_cast<float*>(w + p.unit);
  a.chunk_runs = r.chunk_runs;
  a.tile_runs = r.tile_runs;
  a.unique = g.unique;
  a.dout_ld = g.dout_ld;
  a.seg_pitch = g.seg_pitch;
  a.grad_ld = g.grad_ld;
  a.n = p.n;
  a.rows = s.rows;
  a.cols = s.cols;
  a.ch = p.ch;
  a.chunks = p.chunks;
  a.units = p.units;
  a.dim = g.dim;
  a.pdim = (int32_t)p.pdim;
  a.mode = g.mode;
  a.scale = g.scale;
  a.dout_vec = ((uintptr_t)g.dout % 16 == 0 && g.dout_ld * dout_size % 16 == 0 && g.seg_pitch * dout_size % 16 == 0 &&
                g.seg_pitch >= ((int64_t)g.dim + 3) / 4 * 4)
                   ? 1
                   : 0;
  a.grad_vec = grad_vec;
  a.div_cols = s.div_cols;
  a.group_shift = p.shift;
  return g.grad_f32 ? launch_segments<true>(a, g.dout_f32, stream)
                    : launch_segments<false>(a, g.dout_f32, stream);
}

}  // namespace engram
