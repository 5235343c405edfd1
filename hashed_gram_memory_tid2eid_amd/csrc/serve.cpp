// serve.cpp -- the extern "C" entry points of the serving operators in include/engram.h:
// argument checks that the host can make, then kernel launches on the caller's stream.
// None allocates or synchronises.
#include <hip/hip_runtime.h>

#include "internal.h"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

constexpr int64_t kMax32 = 0x7FFFFFFF;
// workgroups of 256 lanes in one launch: the lanes of a grid are counted in 32 bits
constexpr int64_t kMaxGroups = (1 << 24) - 1;

// Tables of `rows` rows over a pool of num_pages pages of page_size tokens.
int pool_shape(int64_t rows, int64_t table_ld, int32_t max_blocks, int32_t page_size, int32_t num_pages) {
  if (rows < 0 || max_blocks < 0 || table_ld < max_blocks || page_size < 1 || num_pages < 0) return ENGRAM_E_ARG;
  if (num_pages >= 1 << 30 || (int64_t)page_size * max_blocks > kMax32) return ENGRAM_E_UNSUPPORTED;
  return ENGRAM_OK;
}

}  // namespace

extern "C" int engram_block_plan(const int32_t* d_past, const int32_t* d_new, int32_t R, int32_t page_size,
                                 int32_t* d_tables, int64_t table_ld, int32_t max_blocks, const uint32_t* d_free,
                                 uint32_t* d_free_out, int32_t num_pages, int32_t* d_cu_seqlens, uint8_t* d_seq_start,
                                 int32_t* d_lens, int32_t T, int32_t* d_positions, int64_t* d_token_slots,
                                 hipStream_t stream) {
  const int rc = pool_shape(R, table_ld, max_blocks, page_size, num_pages);
  if (rc != ENGRAM_OK) return rc;
  if (T < 0 || !d_cu_seqlens || (T > 0 && !d_token_slots)) return ENGRAM_E_ARG;
  if (R > engram::kPlanMaxRows || T == kMax32) return ENGRAM_E_UNSUPPORTED;
  if (R > 0 && (!d_past || !d_new || (max_blocks > 0 && !d_tables))) return ENGRAM_E_ARG;
  if (num_pages > 0 && (!d_free || !d_free_out)) return ENGRAM_E_ARG;
  if (!aligned(d_past, 4) || !aligned(d_new, 4) || !aligned(d_tables, 4) || !aligned(d_free, 4) ||
      !aligned(d_free_out, 4) || !aligned(d_cu_seqlens, 4) || !aligned(d_lens, 4) || !aligned(d_positions, 4) ||
      !aligned(d_token_slots, 8))
    return ENGRAM_E_ALIGN;
  engram::PlanArgs a = {};
  a.past = d_past;
  a.fresh = d_new;
  a.R = R;
  a.page_size = page_size;
  a.tables = d_tables;
  a.table_ld = table_ld;
  a.max_blocks = max_blocks;
  a.free = d_free;
  a.free_out = d_free_out;
  a.num_pages = num_pages;
  a.cu_seqlens = d_cu_seqlens;
  a.seq_start = d_seq_start;
  a.lens = d_lens;
  a.T = T;
  a.positions = d_positions;
  a.token_slots = d_token_slots;
  return engram::hip_error_status(engram::launch_block_plan(a, stream));
}

extern "C" int engram_block_release(const int32_t* d_tables, int64_t table_ld, int32_t max_blocks,
                                    const int32_t* d_lens, const uint8_t* d_flags, int32_t R, int32_t page_size,
                                    uint32_t* d_free, int32_t num_pages, hipStream_t stream) {
  const int rc = pool_shape(R, table_ld, max_blocks, page_size, num_pages);
  if (rc != ENGRAM_OK) return rc;
  if (R > kMaxGroups) return ENGRAM_E_UNSUPPORTED;
  if (R == 0 || max_blocks == 0) return ENGRAM_OK;
  if (!d_tables || !d_lens || !d_flags || (num_pages > 0 && !d_free)) return ENGRAM_E_ARG;
  if (!aligned(d_tables, 4) || !aligned(d_lens, 4) || !aligned(d_free, 4)) return ENGRAM_E_ALIGN;
  engram::ReleaseArgs a = {};
  a.tables = d_tables;
  a.table_ld = table_ld;
  a.max_blocks = max_blocks;
  a.lens = d_lens;
  a.flags = d_flags;
  a.R = R;
  a.page_size = page_size;
  a.free = d_free;
  a.num_pages = num_pages;
  return engram::hip_error_status(engram::launch_block_release(a, stream));
}

namespace {

int select_shape(int32_t G, int32_t K, int32_t V, int32_t n) {
  if (G < 0 || K < 1 || V < 1 || n < 1) return ENGRAM_E_ARG;
  if (K > 64 || n > 64 || V > 1 << 24 || (int64_t)G * K > 1 << 20) return ENGRAM_E_UNSUPPORTED;
  if ((int64_t)G * K * ((V + 8191) / 8192) > kMaxGroups) return ENGRAM_E_UNSUPPORTED;  // pieces of 8,192 fp32
  return ENGRAM_OK;
}

}  // namespace

extern "C" int engram_beam_select_workspace(int32_t G, int32_t K, int32_t V, int32_t n, int64_t* bytes) {
  if (!bytes) return ENGRAM_E_ARG;
  const int rc = select_shape(G, K, V, n);
  if (rc != ENGRAM_OK) return rc;
  *bytes = engram::beam_select_workspace_bytes(G, K, V, n);
  return ENGRAM_OK;
}

extern "C" int engram_beam_select(const void* d_logits, int32_t logits_dtype, int64_t ld, int32_t G, int32_t K,
                                  int32_t V, const float* d_scores, const uint8_t* d_done, int32_t end_token,
                                  int32_t n, int32_t* d_tokens, int32_t* d_parents, float* d_out_scores,
                                  uint8_t* d_out_done, void* d_work, int64_t work_bytes, hipStream_t stream) {
  if (logits_dtype != ENGRAM_DTYPE_BF16 && logits_dtype != ENGRAM_DTYPE_F32) return ENGRAM_E_ARG;
  const int rc = select_shape(G, K, V, n);
  if (rc != ENGRAM_OK) return rc;
  if (ld < V || end_token < -1 || end_token >= V || (d_done && end_token < 0)) return ENGRAM_E_ARG;
  if (G == 0) return ENGRAM_OK;
  if (!d_logits || !d_scores || !d_tokens || !d_parents || !d_out_scores || !d_work) return ENGRAM_E_ARG;
  if (work_bytes < engram::beam_select_workspace_bytes(G, K, V, n)) return ENGRAM_E_SCRATCH;
  if (!aligned(d_logits, logits_dtype == ENGRAM_DTYPE_F32 ? 4 : 2) || !aligned(d_scores, 4) || !aligned(d_tokens, 4) ||
      !aligned(d_parents, 4) || !aligned(d_out_scores, 4) || !aligned(d_work, 16))
    return ENGRAM_E_ALIGN;
  engram::SelectArgs a = {};
  a.logits = d_logits;
  a.f32 = logits_dtype == ENGRAM_DTYPE_F32;
  a.ld = ld;
  a.G = G;
  a.K = K;
  a.V = V;
  a.scores = d_scores;
  a.done = d_done;
  a.end_token = end_token;
  a.n = n;
  a.tokens = d_tokens;
  a.parents = d_parents;
  a.out_scores = d_out_scores;
  a.out_done = d_out_done;
  a.work = d_work;
  return engram::hip_error_status(engram::launch_beam_select(a, stream));
}

extern "C" int engram_beam_reorder(const int32_t* d_parents, int32_t G, int32_t K, engram_store* store,
                                   const int32_t* d_slots, int32_t* d_slots_out, int32_t* d_slot_src,
                                   int32_t* d_slot_dst, const int32_t* d_tables, int32_t* d_tables_out,
                                   int64_t table_ld, int32_t max_blocks, const int32_t* d_lens, int32_t page_size,
                                   uint32_t* d_free, int32_t num_pages, int32_t* d_page_src, int32_t* d_page_dst,
                                   hipStream_t stream) {
  if (G < 0 || K < 1) return ENGRAM_E_ARG;
  if (K > 64 || (int64_t)G * K > 1 << 20) return ENGRAM_E_UNSUPPORTED;
  if (G == 0) return ENGRAM_OK;  // (arrays without entries may be null)
  if (!d_slots && !d_tables) return ENGRAM_E_ARG;
  if (d_slots ? !d_slots_out : (store || d_slots_out || d_slot_src || d_slot_dst)) return ENGRAM_E_ARG;
  if (store) {
    const int rc = engram::store_usable(store, nullptr);
    if (rc != ENGRAM_OK) return rc;
  }
  if (d_tables) {
    const int rc = pool_shape((int64_t)G * K, table_ld, max_blocks, page_size, num_pages);
    if (rc != ENGRAM_OK) return rc;
    if (!d_tables_out || !d_lens) return ENGRAM_E_ARG;
    const int64_t tiles = ((int64_t)max_blocks + 255) / 256;
    if (tiles > 65535 || tiles * G > kMaxGroups) return ENGRAM_E_UNSUPPORTED;
  } else if (d_tables_out || d_free || d_page_src || d_page_dst) {
    return ENGRAM_E_ARG;
  }
  if (!d_parents) return ENGRAM_E_ARG;
  for (const void* p : {(const void*)d_parents, (const void*)d_slots, (const void*)d_slots_out, (const void*)d_slot_src,
                        (const void*)d_slot_dst, (const void*)d_tables, (const void*)d_tables_out, (const void*)d_lens,
                        (const void*)d_free, (const void*)d_page_src, (const void*)d_page_dst})
    if (!aligned(p, 4)) return ENGRAM_E_ALIGN;
  engram::ReorderArgs a = {};
  a.parents = d_parents;
  a.G = G;
  a.K = K;
  a.store = store ? store->ids : nullptr;
  a.num_slots = store ? store->num_slots : 0;
  a.slots = d_slots;
  a.slots_out = d_slots_out;
  a.slot_src = d_slot_src;
  a.slot_dst = d_slot_dst;
  a.tables = d_tables;
  a.tables_out = d_tables_out;
  a.table_ld = table_ld;
  a.max_blocks = max_blocks;
  a.lens = d_lens;
  a.page_size = page_size;
  a.free = d_free;
  a.num_pages = num_pages;
  a.page_src = d_page_src;
  a.page_dst = d_page_dst;
  return engram::hip_error_status(engram::launch_beam_reorder(a, stream));
}

namespace {

// `count` spans of `bytes`, `pitch` apart, end within `most` (all of them positive).
bool spans_within(int64_t count, int64_t pitch, int64_t bytes, int64_t most) {
  return most >= bytes && (count - 1 == 0 || pitch <= (most - bytes) / (count - 1));
}

// No byte is in two rows: planes whole one behind another, or rows whole with their planes inside.
bool rows_apart(int64_t planes, int64_t plane_pitch, int64_t rows, int64_t row_pitch, int64_t row_bytes) {
  if (planes <= 1 || rows == 0) return true;
  return spans_within(rows, row_pitch, row_bytes, plane_pitch) ||
         (plane_pitch >= row_bytes && spans_within(planes, plane_pitch, row_bytes, row_pitch));
}

}  // namespace

extern "C" int engram_state_copy(void* d_state, int64_t planes, int64_t plane_pitch, int64_t rows, int64_t row_pitch,
                                 int64_t row_bytes, const int32_t* d_src, const int32_t* d_dst, int32_t n,
                                 hipStream_t stream) {
  if (planes < 0 || plane_pitch < 0 || rows < 0 || row_bytes < 1 || row_pitch < row_bytes || n < 0) return ENGRAM_E_ARG;
  if (rows > kMax32 || row_bytes > 65535 * 1024) return ENGRAM_E_UNSUPPORTED;  // that many pieces of single bytes
  if (planes > kMaxGroups || (int64_t)n * planes > kMaxGroups) return ENGRAM_E_UNSUPPORTED;
  if (!rows_apart(planes, plane_pitch, rows, row_pitch, row_bytes)) return ENGRAM_E_ARG;
  if (n == 0 || planes == 0) return ENGRAM_OK;
  if ((!d_state && rows > 0) || !d_src || !d_dst) return ENGRAM_E_ARG;
  if (!aligned(d_src, 4) || !aligned(d_dst, 4)) return ENGRAM_E_ALIGN;
  engram::StateCopyArgs a = {};
  a.state = static_cast<char*>(d_state);
  a.planes = planes;
  a.plane_pitch = plane_pitch;
  a.rows = rows;
  a.row_pitch = row_pitch;
  a.row_bytes = row_bytes;
  a.src = d_src;
  a.dst = d_dst;
  a.n = n;
  return engram::hip_error_status(engram::launch_state_copy(a, stream));
}
