// beam_reorder.hip -- slots, store entries and block tables follow beam search's selection, and
// the copy of the rows that this names.  Included into engram_device.hip after blocks.hip.
//
// Every workgroup works the request's assignment out for itself, a beam a lane: the lanes that
// name beam b are one ballot, whose lowest is b's heir; the other lanes take the beams whose
// ballot is empty, in order.  A block table is then permuted a tile of 256 columns at a time
// through LDS, so that in place and out of place are the same code.  A page of a full block is
// freed where a beam that no row continues names it and no continued one does; both are at the
// same column, which is where beams of one request share pages.  512 requests of 8 beams, 1,024
// blocks: 8.5 us, with store entries 8.6 (slots alone 3.0 and 3.4): the parents and lengths, then
// the columns, then the stores, each waiting for the last.

namespace engram {

constexpr int kReorderColumns = 256;
constexpr int kMaxBeams = 64;

// Pages, slots and pairs of one request.
__global__ __launch_bounds__(kReorderColumns) void beam_reorder_kernel(ReorderArgs a) {
  extern __shared__ int32_t tile[];  // [K][kReorderColumns]
  __shared__ int heir_of[kMaxBeams];    // the beam whose slot and last page child c takes over
  __shared__ int parent_of[kMaxBeams];  // the beam whose full blocks it continues
  __shared__ int lost[kMaxBeams], kept[kMaxBeams];
  __shared__ int num_lost, num_kept, length;
  const int g = blockIdx.x, tid = threadIdx.x, K = a.K;
  const int64_t row0 = (int64_t)g * K;

  if (tid < 64) {
    const bool in = tid < K;
    int parent = in ? a.parents[row0 + tid] : -1;
    const int32_t len = in && a.tables != nullptr ? a.lens[row0 + tid] : 0;
    const int32_t len0 = __shfl(len, 0, 64);
    int fault = 0;
    if (__ballot(parent < -1 || parent >= K) != 0) fault = ENGRAM_E_PARENT_RANGE;
    if (__ballot(in && a.tables != nullptr && (len != len0 || len < 0 || len > (int64_t)a.max_blocks * a.page_size)) != 0)
      fault = ENGRAM_E_SEQLENS;
    if (fault != 0) {
      if (tid == 0 && blockIdx.y == 0) latch_error(fault);
      parent = tid;  // all stay where they are
    }
    const unsigned long long below = (1ull << tid) - 1ull;
    unsigned long long alive = 0, heirs = 0;
    for (int b = 0; b < K; ++b) {
      const unsigned long long children = __ballot(in && parent == b);
      if (children != 0) {
        alive |= 1ull << b;
        heirs |= children & (~children + 1ull);
      }
    }
    const unsigned long long all = K == 64 ? ~0ull : (1ull << K) - 1ull;
    const unsigned long long dead = all & ~alive, others = all & ~heirs;
    const bool is_heir = heirs >> tid & 1ull;
    int heir = is_heir ? parent : tid;
    if (in && !is_heir) {  // as many of these as beams without children
      unsigned long long left = dead;
      for (int skip = __popcll(others & below); skip > 0; --skip) left &= left - 1ull;
      heir = __ffsll(left) - 1;
    }
    const int continued = parent >= 0 ? parent : heir;
    // beams that some row's full blocks continue, and those that none does
    const unsigned long long orphans = __ballot(in && parent < 0);
    unsigned long long named = alive;
    for (unsigned long long o = orphans; o != 0; o &= o - 1ull)
      named |= 1ull << __shfl(heir, __ffsll(o) - 1, 64);
    const unsigned long long gone = all & ~named;
    if (in) {
      heir_of[tid] = heir;
      parent_of[tid] = continued;
      if (gone >> tid & 1ull)
        lost[__popcll(gone & below)] = tid;
      else
        kept[__popcll(named & below)] = tid;
    }
    if (tid == 0) {
      num_lost = __popcll(gone);
      num_kept = __popcll(named);
      length = fault == ENGRAM_E_SEQLENS ? 0 : len0;
    }

    if (blockIdx.y == 0 && a.slots != nullptr) {
      const int32_t own = in ? a.slots[row0 + tid] : -1;
      const int32_t to = __shfl(own, heir, 64), from = __shfl(own, continued, 64);
      const bool pair = in && continued != heir && from >= 0 && to >= 0;
      int32_t ids[3] = {0, 0, 0};
      bool copy = pair && a.store != nullptr;
      if (copy && (from >= a.num_slots || to >= a.num_slots)) {
        latch_error(ENGRAM_E_SLOT_RANGE);
        copy = false;
      }
      if (copy)
        for (int j = 0; j < 3; ++j) ids[j] = a.store[3 * (int64_t)from + j];
      if (in) {
        a.slots_out[row0 + tid] = to;
        if (a.slot_src != nullptr) a.slot_src[row0 + tid] = pair ? from : -1;
        if (a.slot_dst != nullptr) a.slot_dst[row0 + tid] = pair ? to : -1;
      }
      if (copy)
        for (int j = 0; j < 3; ++j) a.store[3 * (int64_t)to + j] = ids[j];
    }
  }
  if (a.tables == nullptr) return;
  __syncthreads();

  const uint32_t P = (uint32_t)a.page_size, len = (uint32_t)length;
  const int full = (int)(len / P), blocks = full + (len % P != 0 ? 1 : 0);
  if (blockIdx.y == 0 && full == blocks && tid < K) {  // no partly filled page
    if (a.page_src != nullptr) a.page_src[row0 + tid] = -1;
    if (a.page_dst != nullptr) a.page_dst[row0 + tid] = -1;
  }
  const int c0 = blockIdx.y * kReorderColumns, col = c0 + tid;
  if (c0 >= blocks) return;
  const int32_t* old = a.tables + row0 * a.table_ld;
  int32_t* out = a.tables_out + row0 * a.table_ld;
  if (col < blocks)
    for (int b = 0; b < K; ++b) tile[b * kReorderColumns + tid] = old[b * a.table_ld + col];
  __syncthreads();  // (for the pairs, which are another lane's column; each lane writes its own)
  if (col < blocks) {
    const int* from = col < full ? parent_of : heir_of;
    for (int c = 0; c < K; ++c) out[c * a.table_ld + col] = tile[from[c] * kReorderColumns + tid];
  }
  if (col < full && a.free != nullptr) {
    for (int i = 0; i < num_lost; ++i) {
      const int32_t page = tile[lost[i] * kReorderColumns + tid];
      bool still = page < 0;
      for (int k = 0; k < num_kept && !still; ++k) still = tile[kept[k] * kReorderColumns + tid] == page;
      if (still) continue;
      if (page >= a.num_pages)
        latch_error(ENGRAM_E_PAGE_RANGE);
      else
        atomicOr(&a.free[page >> 5], 1u << (page & 31));
    }
  }
  if (full < blocks && full >= c0 && full < c0 + kReorderColumns && tid < K) {
    const int at = full - c0;
    const int32_t from = tile[parent_of[tid] * kReorderColumns + at], to = tile[heir_of[tid] * kReorderColumns + at];
    bool pair = parent_of[tid] != heir_of[tid];
    if (pair && (from < 0 || to < 0 || from >= a.num_pages || to >= a.num_pages)) {
      latch_error(ENGRAM_E_PAGE_RANGE);
      pair = false;
    }
    if (a.page_src != nullptr) a.page_src[row0 + tid] = pair ? from : -1;
    if (a.page_dst != nullptr) a.page_dst[row0 + tid] = pair ? to : -1;
  }
}

hipError_t launch_beam_reorder(const ReorderArgs& a, hipStream_t stream) {
  (void)hipGetLastError();  // drop a stale error another library left on this thread
  if (a.G == 0) return hipSuccess;
  const int tiles = a.tables == nullptr ? 1 : std::max(1, (a.max_blocks + kReorderColumns - 1) / kReorderColumns);
  const int lds = a.tables == nullptr ? 0 : a.K * kReorderColumns * (int)sizeof(int32_t);
  static std::atomic<uint64_t> done{0};
  const hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(beam_reorder_kernel),
                                          kMaxBeams * kReorderColumns * (int)sizeof(int32_t), done);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(beam_reorder_kernel, dim3(a.G, tiles), dim3(kReorderColumns), lds, stream, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Rows copied as named: 4 units (of 16, 4 or 1 bytes) a lane, as many lanes a row as its length
// takes, up to a workgroup, which then takes one piece of it; a pair's planes by neighbouring
// workgroups.  Bound by memory: 256 pairs of 16 KB in 32 planes, 268 MB, 51 us (5.3 TB/s).  Plane
// by plane 55; ordinary stores 60; loads past the caches, too, 54; one unit a lane 62; 2,048
// workgroups that go on from item to item 62.  Units of 4 and of 1 byte (one state, part of it in
// the last cache): 46 us for rows of 16,380 bytes, 174 for 16,383, against 37.6 for 16,384.

constexpr int kCopyThreads = 256;
typedef uint32_t copy16_t __attribute__((ext_vector_type(4)));

template <typename U>
__global__ __launch_bounds__(kCopyThreads) void state_copy_kernel(StateCopyArgs a, uint32_t units, uint32_t lanes) {
  // `lanes` lanes share one (pair, plane); blockIdx.y counts pieces of kCopyThreads * 4 units
  const uint32_t per = kCopyThreads / lanes;
  const uint64_t item = (uint64_t)blockIdx.x * per + threadIdx.x / lanes;
  const uint64_t items = (uint64_t)a.n * (uint64_t)a.planes;
  if (item >= items) return;
  const int64_t pair = (int64_t)(item / (uint32_t)a.planes), plane = (int64_t)(item % (uint32_t)a.planes);
  const int32_t src = a.src[pair], dst = a.dst[pair];
  if (src == -1 || dst == -1 || src == dst) return;
  if (src < 0 || dst < 0 || src >= a.rows || dst >= a.rows) {
    latch_error(ENGRAM_E_SLOT_RANGE);
    return;
  }
  const U* from = reinterpret_cast<const U*>(a.state + plane * a.plane_pitch + src * a.row_pitch);
  U* to = reinterpret_cast<U*>(a.state + plane * a.plane_pitch + dst * a.row_pitch);
  const uint32_t first = blockIdx.y * lanes * 4 + threadIdx.x % lanes;
  U v[4];
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j)
    if (first + j * lanes < units) v[j] = from[first + j * lanes];
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j)
    if (first + j * lanes < units) __builtin_nontemporal_store(v[j], to + first + j * lanes);
}

hipError_t launch_state_copy(const StateCopyArgs& a, hipStream_t stream) {
  (void)hipGetLastError();  // drop a stale error another library left on this thread
  if (a.n == 0 || a.planes == 0) return hipSuccess;
  const uintptr_t all = (uintptr_t)a.state | (uintptr_t)a.plane_pitch | (uintptr_t)a.row_pitch | (uintptr_t)a.row_bytes;
  const int unit = all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 1;
  const uint32_t units = (uint32_t)(a.row_bytes / unit);
  uint32_t lanes = 1;
  while (lanes < (uint32_t)kCopyThreads && lanes * 4 < units) lanes <<= 1;
  const uint64_t items = (uint64_t)a.n * (uint64_t)a.planes, per = kCopyThreads / lanes;
  const dim3 grid((unsigned)((items + per - 1) / per), (units + lanes * 4 - 1) / (lanes * 4));
  if (unit == 16)
    hipLaunchKernelGGL(state_copy_kernel<copy16_t>, grid, dim3(kCopyThreads), 0, stream, a, units, lanes);
  else if (unit == 4)
    hipLaunchKernelGGL(state_copy_kernel<uint32_t>, grid, dim3(kCopyThreads), 0, stream, a, units, lanes);
  else
    hipLaunchKernelGGL(state_copy_kernel<uint8_t>, grid, dim3(kCopyThreads), 0, stream, a, units, lanes);
  return hipGetLastError();
}

}  // namespace engram
