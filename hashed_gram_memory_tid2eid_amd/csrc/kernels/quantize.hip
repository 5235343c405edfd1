// quantize.hip -- blocks of 128 values to OCP e4m3fn codes with one scale each: the operands
// of gemm_fp8.hip.  Included into engram_device.hip.
//
//   s = max(fl32(amax / 448), 2^-126), or the least power of two not below that (e8m0)
//   code = e4m3fn(fl32(x / s)), nearest even;  |x / s| <= 448 (1 + 2^-24), so nothing overflows
//
// Blocks are 1 x 128 along the rows (codes [M][K], scales [K / 128][M]), 1 x 128 along the
// columns (the transposed codes [K][M], scales [M / 128][K]), both in one pass over x, or
// 128 x 128 (one scale, both codes).  Codes past the matrix, up to whole blocks, are zero.
// The largest magnitude is taken as an unsigned maximum of the bits, so that a NaN wins: a
// block that holds an infinity or a NaN becomes all NaN.
//
// The quotient without a division per element: r = fl(1 / s) once per block, y = fl(x r),
// and one correction y + (x - y s) r with the residual exact in an fma.  With r correctly
// rounded this is the correctly rounded quotient (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990).  The residual has to stay clear of
// the end of fp32: a wave that meets a scale under 2^-64 does its codes once more, with x and s
// both 2^64 times as large (left as they are, 4 to 6% of the quotients that lie on a tie gave
// the other code for s around 2^-122).
//
// A workgroup of 4 waves holds a tile of 16 RT rows x 128 columns in registers: lane l of
// wave w holds 8 consecutive columns (l % 16) of RT consecutive rows, so a wave's loads are
// whole lines, a row's maximum is a reduction over 16 lanes, and a column's one over the
// thread's own rows, 4 lanes and 4 waves.  Transposed codes of a thread are 8 rows = 8 bytes
// of a column; they cross LDS (16 KB) and leave as 128-byte lines.
//
// Memory bounds it.  Codes are written past the caches (16,381 x 4,096 fp32 both ways 72 us
// against 84): 407 MB in 74 us, 5.5 TB/s; 16,381 x 6,144 bf16 both ways 88 us, 4.7 TB/s; 65,536 x
// 6,144 bf16 rows alone 210 us (5.8 TB/s), both ways 423 us (3.9 TB/s: every tile of the
// transposed codes is 128 lines that lie 64 KB apart); 4,096 x 6,144 fp32 in blocks of 128 x 128,
// both codes, 23 us (6.6 TB/s, x in the last cache).  An order of the tiles that keeps those lines together (4 to 32 rows of tiles
// at a time) measured the same.

namespace engram {

constexpr int kQuantThreads = 256;
constexpr float kE4m3Max = 448.0f;
constexpr float kQuantUp = 0x1p64f;  // what x and s of a small block are multiplied by

struct QuantScale {
  float s, r;       // the scale and its reciprocal
  uint32_t held;    // float bits, or the e8m0 byte
};

template <bool E8M0>
__device__ __forceinline__ QuantScale quant_scale(uint32_t amax_bits) {
  const float q = __uint_as_float(amax_bits) / kE4m3Max;
  const float c = q < 0x1p-126f ? 0x1p-126f : q;  // keeps a NaN
  QuantScale o;
  if (E8M0) {
    const uint32_t b = __float_as_uint(c);
    const uint32_t e = min((b >> 23) + ((b & 0x7FFFFFu) != 0 ? 1u : 0u), 255u);
    o.held = e;
    o.s = e == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(e << 23);
    // 2^(127 - e): e = 254 needs the subnormal 2^-127
    o.r = e == 255u ? o.s : (e == 254u ? __uint_as_float(0x00400000u) : __uint_as_float((254u - e) << 23));
  } else {
    o.held = __float_as_uint(c);
    o.s = c;
    o.r = 1.0f / c;
  }
  return o;
}

// whether a float scale is too small for quotients as they are: under 2^-64, but not 2^-126, which
// divides exactly (and is the scale of every empty block)
__device__ __forceinline__ bool quant_small(const QuantScale& q) { return q.held - 0x00800001u < 0x1F800000u - 0x00800001u; }

template <bool E8M0, bool SMALL>
__device__ __forceinline__ float quant_quotient(float x, const QuantScale& q) {
  if (SMALL && quant_small(q)) {
    const float v = x * kQuantUp, s = q.s * kQuantUp, r = q.r * (1.0f / kQuantUp), y = v * r;
    return fmaf(fmaf(-y, s, v), r, y);
  }
  const float y = x * q.r;
  if (E8M0) return y;  // a power of two: exact
  return fmaf(fmaf(-y, q.s, x), q.r, y);
}

// four codes in one word, the first in the low byte
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

struct QuantKArgs {
  const void* x;
  uint8_t* q;
  uint8_t* qt;
  void* s;
  void* st;
  int64_t ld, q_ld, qt_ld;
  int32_t M, K, KB, MB;  // KB, MB: blocks of 128 along k, along m
  int32_t vec;           // x rows start on 16 bytes
};

// LDS slot (8 bytes) of column `col`, row group g (8 rows): the groups of a column are
// permuted by its 8-column block, which spreads a wave's writes over the banks
__device__ __forceinline__ int quant_slot(int col, int g) { return col * 16 + (g ^ ((col >> 3) & 15)); }

// (tiles of 128 rows: three waves a SIMD; left alone the compiler takes registers for two, and
// 16,381 x 6,144 bf16 both ways took 103 us where three took 80; four spill.  The transpose alone
// fits five)
template <bool X_F32, bool E8M0, bool ROWS, bool COLS, bool BLOCK, int RT>
__global__ __launch_bounds__(kQuantThreads, RT < 8 ? 1 : ROWS || BLOCK ? 3 : 5) void fp8_quantize_kernel(QuantKArgs a) {
  static_assert(!(COLS || BLOCK) || RT == 8, "column blocks need a tile of 128 rows");
  constexpr int TILE_M = 16 * RT;
  __shared__ uint64_t tile[COLS ? 128 * 16 : 1];
  __shared__ uint32_t colmax[(COLS || BLOCK) ? 4 : 1][128];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int kb = blockIdx.x % (uint32_t)a.KB;
  const int mt = blockIdx.x / (uint32_t)a.KB;
  const int c = lane & 15;
  const int k0 = kb * 128 + c * 8;
  const int64_t m0 = (int64_t)mt * TILE_M;
  const int r0 = wave * (4 * RT) + (lane >> 4) * RT;  // first of the thread's rows in the tile
  const int nk = min(8, a.K - k0);                    // columns of the thread inside the matrix

  float x[RT][8];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t m = m0 + r0 + i;
    if (m < a.M && nk > 0) {
      load_chunk<X_F32, 8>(a.x, m * a.ld + k0, nk, a.vec != 0, x[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = 0.0f;
    }
  }

  uint32_t block_max = 0;
  if constexpr (COLS || BLOCK) {
    uint32_t cm[8] = {};
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) cm[j] = max(cm[j], __float_as_uint(x[i][j]) & 0x7FFFFFFFu);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      cm[j] = max(cm[j], (uint32_t)__shfl_xor((int)cm[j], 16, 64));
      cm[j] = max(cm[j], (uint32_t)__shfl_xor((int)cm[j], 32, 64));
    }
    if (lane < 16) {
#pragma unroll
      for (int j = 0; j < 8; ++j) colmax[wave][c * 8 + j] = cm[j];
    }
    __syncthreads();
    if (BLOCK) {
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int h = 0; h < 2; ++h) block_max = max(block_max, colmax[w][h * 64 + lane]);
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) block_max = max(block_max, (uint32_t)__shfl_xor((int)block_max, off, 64));
    }
  }
  QuantScale one = {};
  if (BLOCK) {
    one = quant_scale<E8M0>(block_max);
    if (!E8M0 && quant_small(one)) {  // uniform
      one.s *= kQuantUp;
      one.r *= 1.0f / kQuantUp;
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] *= kQuantUp;
    }
    if (tid == 0) {
      if (ROWS) {
        const int64_t at = (int64_t)kb * a.MB + mt;
        if (E8M0) static_cast<uint8_t*>(a.s)[at] = (uint8_t)one.held;
        else static_cast<uint32_t*>(a.s)[at] = one.held;
      }
      if (COLS) {
        const int64_t at = (int64_t)mt * a.KB + kb;
        if (E8M0) static_cast<uint8_t*>(a.st)[at] = (uint8_t)one.held;
        else static_cast<uint32_t*>(a.st)[at] = one.held;
      }
    }
  }

  // the codes along the rows; returns whether a scale of the thread's is small
  auto row_codes = [&](auto careful) -> bool {
    bool small = false;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int64_t m = m0 + r0 + i;
      if (careful()) __builtin_amdgcn_sched_barrier(0);  // one row after the other, in few registers
      QuantScale q = one;
      if (!BLOCK) {
        uint32_t rm = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) rm = max(rm, __float_as_uint(x[i][j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) rm = max(rm, (uint32_t)__shfl_xor((int)rm, off, 64));
        q = quant_scale<E8M0>(rm);
        small |= quant_small(q);
      }
      if (m >= a.M) continue;
      if (!BLOCK && c == 0) {
        const int64_t at = (int64_t)kb * a.M + m;
        if (E8M0) static_cast<uint8_t*>(a.s)[at] = (uint8_t)q.held;
        else static_cast<uint32_t*>(a.s)[at] = q.held;
      }
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = quant_quotient<E8M0, careful()>(x[i][j], q);
      uint2 o;
      o.x = pack_e4m3x4(y[0], y[1], y[2], y[3]);
      o.y = pack_e4m3x4(y[4], y[5], y[6], y[7]);
      __builtin_nontemporal_store((uint64_t)o.x | ((uint64_t)o.y << 32), reinterpret_cast<uint64_t*>(a.q + m * a.q_ld + k0));
    }
    return small;
  };
  if constexpr (ROWS) {
    const bool small = row_codes(std::false_type());
    if (!E8M0 && !BLOCK && __any(small)) row_codes(std::true_type());
  }

  // the codes along the columns, into LDS
  auto column_codes = [&](auto careful) -> bool {
    bool small = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = c * 8 + j;
      if (careful()) __builtin_amdgcn_sched_barrier(0);
      QuantScale q = one;
      if (!BLOCK) {
        const uint32_t m4 = max(max(colmax[0][col], colmax[1][col]), max(colmax[2][col], colmax[3][col]));
        q = quant_scale<E8M0>(m4);
        small |= quant_small(q);
        if (wave == 0 && lane < 16 && k0 + j < a.K) {
          const int64_t at = (int64_t)mt * a.K + k0 + j;
          if (E8M0) static_cast<uint8_t*>(a.st)[at] = (uint8_t)q.held;
          else static_cast<uint32_t*>(a.st)[at] = q.held;
        }
      }
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = quant_quotient<E8M0, careful()>(x[i % RT][j], q);
      const uint64_t lo = pack_e4m3x4(y[0], y[1], y[2], y[3]), hi = pack_e4m3x4(y[4], y[5], y[6], y[7]);
      tile[quant_slot(col, r0 >> 3)] = lo | (hi << 32);
    }
    return small;
  };
  if constexpr (COLS) {
    const bool small = column_codes(std::false_type());
    if (!E8M0 && !BLOCK && __any(small)) column_codes(std::true_type());
    __syncthreads();
    // 8 lanes write one column's 128 codes: thread -> column tid / 8 + 32 p, 16 bytes tid % 8
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int col = p * 32 + (tid >> 3), part = tid & 7;
      const int64_t k = (int64_t)kb * 128 + col;
      if (k >= a.K) continue;
      const uint64_t lo = tile[quant_slot(col, 2 * part)], hi = tile[quant_slot(col, 2 * part + 1)];
      const u32x4 o = {(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
      __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(a.qt + k * a.qt_ld + m0 + part * 16));
    }
  }
}

template <bool X_F32, bool E8M0>
static void quantize_dispatch(const QuantizeArgs& g, const QuantKArgs& a, hipStream_t stream) {
  const dim3 block(kQuantThreads);
  const dim3 grid((unsigned)((int64_t)a.KB * a.MB));
  const bool rows = g.q != nullptr, cols = g.qt != nullptr;
  if (g.block == 128) {
    if (rows && cols)
      hipLaunchKernelGGL((fp8_quantize_kernel<X_F32, E8M0, true, true, true, 8>), grid, block, 0, stream, a);
    else if (rows)
      hipLaunchKernelGGL((fp8_quantize_kernel<X_F32, E8M0, true, false, true, 8>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((fp8_quantize_kernel<X_F32, E8M0, false, true, true, 8>), grid, block, 0, stream, a);
  } else if (rows && cols) {
    hipLaunchKernelGGL((fp8_quantize_kernel<X_F32, E8M0, true, true, false, 8>), grid, block, 0, stream, a);
  } else if (cols) {
    hipLaunchKernelGGL((fp8_quantize_kernel<X_F32, E8M0, false, true, false, 8>), grid, block, 0, stream, a);
  } else if ((int64_t)a.KB * ((a.M + 31) / 32) <= 2048) {
    // rows alone and few of them: 16 rows a workgroup, so that they spread over the chip
    const dim3 small((unsigned)((int64_t)a.KB * ((a.M + 15) / 16)));
    hipLaunchKernelGGL((fp8_quantize_kernel<X_F32, E8M0, true, false, false, 1>), small, block, 0, stream, a);
  } else {
    const dim3 half((unsigned)((int64_t)a.KB * ((a.M + 63) / 64)));
    hipLaunchKernelGGL((fp8_quantize_kernel<X_F32, E8M0, true, false, false, 4>), half, block, 0, stream, a);
  }
}

hipError_t launch_fp8_quantize(const QuantizeArgs& g, hipStream_t stream) {
  (void)hipGetLastError();
  if (g.M == 0 || g.K == 0) return hipSuccess;
  QuantKArgs a;
  a.x = g.x;
  a.q = g.q;
  a.qt = g.qt;
  a.s = g.s;
  a.st = g.st;
  a.ld = g.ld;
  a.q_ld = g.q_ld;
  a.qt_ld = g.qt_ld;
  a.M = (int32_t)g.M;
  a.K = (int32_t)g.K;
  a.KB = (int32_t)((g.K + 127) / 128);
  a.MB = (int32_t)((g.M + 127) / 128);
  if ((int64_t)a.KB * ((g.M + 15) / 16) > 0x7FFFFFFF) return hipErrorInvalidValue;
  a.vec = ((uintptr_t)g.x % 16 == 0 && g.ld * (g.x_f32 ? 4 : 2) % 16 == 0) ? 1 : 0;
  if (g.x_f32) {
    if (g.e8m0) quantize_dispatch<true, true>(g, a, stream);
    else quantize_dispatch<true, false>(g, a, stream);
  } else {
    if (g.e8m0) quantize_dispatch<false, true>(g, a, stream);
    else quantize_dispatch<false, false>(g, a, stream);
  }
  return hipGetLastError();
}

}  // namespace engram
