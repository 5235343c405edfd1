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
// write past the caches, which then keep table rows instead.  65,536 x 24 rows of 256 bf16
// (Zipf ids, 4M rows, 805 MB written and some 140 MB of distinct rows): 157 us where the rows
// are in the last cache (with ordinary stores 272), 246 us where they come from memory; fp32
// output 264 (464) and 421.  Uniform ids read as much as they write, 1.6 GB in 266 us, 6.1 TB/s;
// that the Zipf ids' 940 MB take 246 is neither their bytes nor their number of requests, and
// is not explained.  In the order 8, 2, 1
// chunks in flight 259, 257, 304 us from memory; rows read past the caches 282.

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

// N elements of a table row as they are loaded, and as floats
template <bool F32, int N>
struct RowChunk {
  static constexpr int WORDS = F32 ? N : N / 2;
  uint32_t w[WORDS];
  __device__ __forceinline__ void load(const void* base, int64_t e, int n, bool vec) {
    if (vec && n == N) {
      typedef uint32_t words __attribute__((ext_vector_type(WORDS < 4 ? WORDS : 4)));
      constexpr int PER = WORDS < 4 ? WORDS : 4;
      const words* src = reinterpret_cast<const words*>(static_cast<const char*>(base) + e * (F32 ? 4 : 2));
#pragma unroll
      for (int h = 0; h < WORDS / PER; ++h) {
        const words v = src[h];
#pragma unroll
        for (int i = 0; i < PER; ++i) w[PER * h + i] = v[i];
      }
    } else {
      float f[N];
      load_chunk<F32, N>(base, e, n, false, f);
#pragma unroll
      for (int i = 0; i < WORDS; ++i)
        w[i] = F32 ? __float_as_uint(f[F32 ? i : 0])
                   : (__float_as_uint(f[F32 ? 0 : 2 * i]) >> 16) | __float_as_uint(f[F32 ? 0 : 2 * i + 1]);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ float at(int i) const {
    if (F32) return __uint_as_float(w[F32 ? i : 0]);
    const uint32_t v = w[F32 ? 0 : i / 2];
    return __uint_as_float(i % 2 ? v & 0xFFFF0000u : v << 16);
  }
};

template <bool TABLE_F32, bool OUT_F32, int UNROLL>
__global__ __launch_bounds__(kEmbedThreads) void embed_kernel(EmbedKArgs a) {
  constexpr int N = OUT_F32 ? 4 : 8;  // elements per chunk
  const uint32_t first = blockIdx.x * (kEmbedThreads * UNROLL) + threadIdx.x;
  // all ids, then all rows: a wait for an id that was asked for behind a row waits for the row, too
  int32_t row[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const uint32_t seg = fdiv(min(first + (uint32_t)u * kEmbedThreads, a.total - 1), a.div_chunks);  // token * cols + column
    const uint32_t t = fdiv(seg, a.div_cols);
    row[u] = a.ids[(int64_t)t * a.ids_ld + (seg - t * a.cols)];
  }
  RowChunk<TABLE_F32, N> raw[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const uint32_t g = min(first + (uint32_t)u * kEmbedThreads, a.total - 1);
    const int e0 = (int)(g - fdiv(g, a.div_chunks) * a.chunks) * N;
    raw[u].clear();
    if (row[u] < 0 || row[u] >= a.rows) {
      if (row[u] != -1) latch_error(ENGRAM_E_ROW_RANGE);
    } else if (e0 < a.dim) {
      raw[u].load(a.table, (int64_t)row[u] * a.table_ld + e0, min(N, a.dim - e0), a.table_vec != 0);
    }
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const uint32_t g = first + (uint32_t)u * kEmbedThreads;
    if (g >= a.total) continue;
    const uint32_t seg = fdiv(g, a.div_chunks), t = fdiv(seg, a.div_cols);
    const int e0 = (int)(g - seg * a.chunks) * N;
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = raw[u].at(i) * a.scale;
    store_chunk<OUT_F32, N, (UNROLL > 1)>(a.out, (int64_t)t * a.out_ld + (int64_t)(seg - t * a.cols) * a.seg_pitch + e0,
                                          (int)min((int64_t)N, a.seg_pitch - e0), a.out_vec != 0, f);
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
