// embed.hip -- the trainable lookup: rows of a bf16 or fp32 table, scaled, into the
// segments of a token row.  Included into engram_device.hip after gather.hip, whose
// helpers it uses.
//
//   out[t][c seg_pitch + d] = scale * table[ids[t][c]][d],  d < dim;  zeros up to seg_pitch
//
// One rounding: the product is fp32 and is rounded to the output's type once (an fp32
// output is the fp32 product).  An id of -1 gives a row of zeros; any other id outside the
// table latches ENGRAM_E_ROW_RANGE and gives zeros too.
//
// The work is a flat list of 8-element output chunks; consecutive lanes take consecutive
// chunks, so a wave's loads and stores are runs of whole cache lines.  Each lane first
// fetches the ids of its UNROLL chunks, then all their table bytes, then stores: that many
// independent row reads are in flight per lane.

namespace engram {

constexpr int kEmbedThreads = 256;

struct EmbedKArgs {
  const void* table;
  const int32_t* ids;
  void* out;
  int64_t rows, table_ld, ids_ld, out_ld, seg_pitch;
  uint32_t total, chunks, cols;  // chunks of 8 in the launch; per segment; segments per token
  int32_t dim;
  float scale;
  int32_t table_vec;  // rows start on 16 bytes: whole chunks load as vectors
  int32_t out_vec;    // segments start on 16 bytes
  FastDiv div_chunks, div_cols;
};

template <bool F32>
__device__ __forceinline__ void load_chunk8(const void* base, int64_t e, int n, bool vec, float* f) {
  if (vec && n == 8) {
    if (F32) {
      const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + e);
      const f32x4 lo = p[0], hi = p[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = lo[i];
        f[4 + i] = hi[i];
      }
    } else {
      const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const unsigned short*>(base) + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[i] = 0.0f;
      if (i < n)
        f[i] = F32 ? static_cast<const float*>(base)[e + i]
                   : __uint_as_float((uint32_t) static_cast<const unsigned short*>(base)[e + i] << 16);
    }
  }
}

template <bool F32>
__device__ __forceinline__ void store_chunk8(void* base, int64_t e, int n, bool vec, const float* f) {
  if (vec && n == 8) {
    if (F32) {
      f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(base) + e);
      p[0] = f32x4{f[0], f[1], f[2], f[3]};
      p[1] = f32x4{f[4], f[5], f[6], f[7]};
    } else {
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = bf16_bits_rne(f[2 * i]) | (bf16_bits_rne(f[2 * i + 1]) << 16);
      *reinterpret_cast<u32x4*>(static_cast<unsigned short*>(base) + e) = o;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if (F32) static_cast<float*>(base)[e + i] = f[i];
        else static_cast<unsigned short*>(base)[e + i] = (unsigned short)bf16_bits_rne(f[i]);
      }
  }
}

template <bool TABLE_F32, bool OUT_F32, int UNROLL>
__global__ __launch_bounds__(kEmbedThreads) void embed_kernel(EmbedKArgs a) {
  const uint32_t first = blockIdx.x * (kEmbedThreads * UNROLL) + threadIdx.x;
  float f[UNROLL][8];
  int64_t dst[UNROLL];
  int n[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const uint32_t g = first + (uint32_t)u * kEmbedThreads;
    n[u] = 0;
    dst[u] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[u][i] = 0.0f;
    if (g >= a.total) continue;
    const uint32_t seg = fdiv(g, a.div_chunks);  // token * cols + column
    const uint32_t chunk = g - seg * a.chunks;
    const uint32_t t = fdiv(seg, a.div_cols);
    const uint32_t c = seg - t * a.cols;
    const int e0 = (int)chunk * 8;
    n[u] = (int)min((int64_t)8, a.seg_pitch - e0);
    dst[u] = (int64_t)t * a.out_ld + (int64_t)c * a.seg_pitch + e0;
    const int32_t row = a.ids[(int64_t)t * a.ids_ld + c];
    if (row < 0 || row >= a.rows) {
      if (row != -1) latch_error(ENGRAM_E_ROW_RANGE);
      continue;
    }
    if (e0 >= a.dim) continue;
    load_chunk8<TABLE_F32>(a.table, (int64_t)row * a.table_ld + e0, min(8, a.dim - e0), a.table_vec != 0, f[u]);
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    if (n[u] == 0) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[u][i] *= a.scale;
    store_chunk8<OUT_F32>(a.out, dst[u], n[u], a.out_vec != 0, f[u]);
  }
}

template <int UNROLL>
static void embed_dispatch(const EmbedArgs& g, const EmbedKArgs& a, dim3 grid, hipStream_t stream) {
  const dim3 block(kEmbedThreads);
  if (g.table_f32 && g.out_f32)
    hipLaunchKernelGGL((embed_kernel<true, true, UNROLL>), grid, block, 0, stream, a);
  else if (g.table_f32)
    hipLaunchKernelGGL((embed_kernel<true, false, UNROLL>), grid, block, 0, stream, a);
  else if (g.out_f32)
    hipLaunchKernelGGL((embed_kernel<false, true, UNROLL>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((embed_kernel<false, false, UNROLL>), grid, block, 0, stream, a);
}

hipError_t launch_embed(const EmbedArgs& g, hipStream_t stream) {
  (void)hipGetLastError();
  if (g.T == 0 || g.cols == 0) return hipSuccess;
  const int64_t chunks = (g.seg_pitch + 7) / 8;
  const int64_t per_token = chunks * g.cols;
  if (per_token > 0x7FFFFFFF) return hipErrorInvalidValue;
  const int64_t max_tokens = (int64_t)0x7FFFFFFF / per_token;  // one launch: fewer than 2^31 chunks
  const size_t out_size = g.out_f32 ? 4 : 2, table_size = g.table_f32 ? 4 : 2;
  EmbedKArgs a;
  a.table = g.table;
  a.rows = g.rows;
  a.table_ld = g.table_ld;
  a.ids_ld = g.ids_ld;
  a.out_ld = g.out_ld;
  a.seg_pitch = g.seg_pitch;
  a.chunks = (uint32_t)chunks;
  a.cols = (uint32_t)g.cols;
  a.dim = g.dim;
  a.scale = g.scale;
  a.table_vec = ((uintptr_t)g.table % 16 == 0 && g.table_ld * table_size % 16 == 0) ? 1 : 0;
  a.out_vec = ((uintptr_t)g.out % 16 == 0 && g.out_ld * out_size % 16 == 0 && g.seg_pitch * out_size % 16 == 0) ? 1 : 0;
  a.div_chunks = make_fastdiv(a.chunks);
  a.div_cols = make_fastdiv(a.cols);
  for (int64_t t0 = 0; t0 < g.T; t0 += max_tokens) {
    const int64_t tn = g.T - t0 < max_tokens ? g.T - t0 : max_tokens;
    a.ids = g.ids + t0 * g.ids_ld;
    a.out = static_cast<char*>(g.out) + (size_t)(t0 * g.out_ld) * out_size;
    a.total = (uint32_t)(tn * per_token);
    // small calls: one chunk per lane, spread over as many workgroups as there are
    if (a.total <= 1024u * kEmbedThreads)
      embed_dispatch<1>(g, a, dim3((a.total + kEmbedThreads - 1) / kEmbedThreads), stream);
    else
      embed_dispatch<4>(g, a, dim3((a.total + 4 * kEmbedThreads - 1) / (4 * kEmbedThreads)), stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace engram
