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
// The work is a flat list of output chunks of 16 bytes (8 bf16 or 4 fp32 elements);
// consecutive lanes take consecutive chunks, so a wave's loads and stores are runs of whole
// cache lines.  Each lane first fetches the ids of its UNROLL chunks, then all their table
// bytes, then stores: that many independent row reads are in flight per lane.  Large calls
// write past the caches, which then keep table rows instead: 65,536 x 24 rows of 256 bf16
// (Zipf ids, 4M rows) 172 us against 289 with ordinary stores (805 MB written), fp32 output
// 290 against 490.  With 2 or 1 chunks in flight 176 and 190 us, with 8 (registers) 224.

namespace engram {

constexpr int kEmbedThreads = 256;
constexpr int kEmbedUnroll = 4;
// calls of up to this many chunks run one chunk per lane, and leave their output cached
constexpr uint32_t kEmbedSmall = 1024 * kEmbedThreads;

struct EmbedKArgs {
  const void* table;
  const int32_t* ids;
  void* out;
  int64_t rows, table_ld, ids_ld, out_ld, seg_pitch;
  uint32_t total, chunks, cols;  // chunks in the launch; per segment; segments per token
  int32_t dim;
  float scale;
  int32_t table_vec;  // rows start on 16 bytes: whole chunks load as vectors
  int32_t out_vec;    // segments start on 16 bytes
  FastDiv div_chunks, div_cols;
};

// N (4 or 8) elements from element e on, the first n of them there; vec: aligned to N elements
template <bool F32, int N>
__device__ __forceinline__ void load_chunk(const void* base, int64_t e, int n, bool vec, float* f) {
  if (vec && n == N) {
    if (F32) {
#pragma unroll
      for (int h = 0; h < N / 4; ++h) {
        const f32x4 v = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + e)[h];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[4 * h + i] = v[i];
      }
    } else {
      uint32_t w[N / 2];
      const unsigned short* src = static_cast<const unsigned short*>(base) + e;
      if (N == 8) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(src);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = v[i];
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(src);
        w[0] = v.x;
        w[1] = v.y;
      }
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      f[i] = 0.0f;
      if (i < n)
        f[i] = F32 ? static_cast<const float*>(base)[e + i]
                   : __uint_as_float((uint32_t) static_cast<const unsigned short*>(base)[e + i] << 16);
    }
  }
}

// NT: written past the caches
template <bool F32, int N, bool NT>
__device__ __forceinline__ void store_chunk(void* base, int64_t e, int n, bool vec, const float* f) {
  if (vec && n == N) {
    if (F32) {
#pragma unroll
      for (int h = 0; h < N / 4; ++h) {
        const f32x4 v = {f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]};
        f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(base) + e) + h;
        if (NT) __builtin_nontemporal_store(v, p);
        else *p = v;
      }
    } else {
      typedef uint32_t words __attribute__((ext_vector_type(N / 2)));
      words o;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) o[i] = bf16_bits_rne(f[2 * i]) | (bf16_bits_rne(f[2 * i + 1]) << 16);
      words* p = reinterpret_cast<words*>(static_cast<unsigned short*>(base) + e);
      if (NT) __builtin_nontemporal_store(o, p);
      else *p = o;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) {
        if (F32) static_cast<float*>(base)[e + i] = f[i];
        else static_cast<unsigned short*>(base)[e + i] = (unsigned short)bf16_bits_rne(f[i]);
      }
  }
}

template <bool TABLE_F32, bool OUT_F32, int UNROLL>
__global__ __launch_bounds__(kEmbedThreads) void embed_kernel(EmbedKArgs a) {
  constexpr int N = OUT_F32 ? 4 : 8;  // elements per chunk
  const uint32_t first = blockIdx.x * (kEmbedThreads * UNROLL) + threadIdx.x;
  float f[UNROLL][N];
  int64_t dst[UNROLL];
  int n[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const uint32_t g = first + (uint32_t)u * kEmbedThreads;
    n[u] = 0;
    dst[u] = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) f[u][i] = 0.0f;
    if (g >= a.total) continue;
    const uint32_t seg = fdiv(g, a.div_chunks);  // token * cols + column
    const uint32_t chunk = g - seg * a.chunks;
    const uint32_t t = fdiv(seg, a.div_cols);
    const uint32_t c = seg - t * a.cols;
    const int e0 = (int)chunk * N;
    n[u] = (int)min((int64_t)N, a.seg_pitch - e0);
    dst[u] = (int64_t)t * a.out_ld + (int64_t)c * a.seg_pitch + e0;
    const int32_t row = a.ids[(int64_t)t * a.ids_ld + c];
    if (row < 0 || row >= a.rows) {
      if (row != -1) latch_error(ENGRAM_E_ROW_RANGE);
      continue;
    }
    if (e0 >= a.dim) continue;
    load_chunk<TABLE_F32, N>(a.table, (int64_t)row * a.table_ld + e0, min(N, a.dim - e0), a.table_vec != 0, f[u]);
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    if (n[u] == 0) continue;
#pragma unroll
    for (int i = 0; i < N; ++i) f[u][i] *= a.scale;
    store_chunk<OUT_F32, N, (UNROLL > 1)>(a.out, dst[u], n[u], a.out_vec != 0, f[u]);
  }
}

template <int UNROLL>
static void embed_dispatch(const EmbedArgs& g, const EmbedKArgs& a, hipStream_t stream) {
  constexpr uint32_t per = kEmbedThreads * UNROLL;
  const dim3 block(kEmbedThreads), grid((a.total + per - 1) / per);
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
  const int64_t per_chunk = g.out_f32 ? 4 : 8;
  const int64_t chunks = (g.seg_pitch + per_chunk - 1) / per_chunk;
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
    if (a.total <= kEmbedSmall) embed_dispatch<1>(g, a, stream);
    else embed_dispatch<kEmbedUnroll>(g, a, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace engram
