// gemm_fp8.hip -- C = A B^T for e4m3fn operands with a scale for each block of 128 along k.
// Included into engram_device.hip after gemm.hip and quantize.hip, whose helpers it uses.
//
//   C[m][n] = sum_kb sa[kb][m] sb[kb][n or n / 128] sum_{k in block kb} A[m][k] B[n][k]
//
// Two matrix instructions, by the type of C:
// - bf16 C: v_mfma_f32_16x16x128_f8f6f4 on the codes; one instruction is one k block of a
//   16 x 16 tile.  It adds the products of a lane's neighbouring codes with some 16 bits
//   below the largest (random codes: 1.4e-5 of the result, in the 2-norm, at any K), which is
//   far below a bf16 step.
// - fp32 C: the codes are widened to bf16 in registers, exactly, and multiplied by
//   v_mfma_f32_16x16x32_bf16, whose sums keep fp32 (1e-7 at K = 6,144), at half the rate.
//   The 8-bit instruction of that shape (16x16x32) has this rate and the short sums.
//
// A lane's operand is 32 codes of one row; which 32 of the block's 128 does not matter as
// long as both operands agree (the scale is one for all 128), so a lane takes 16-byte chunks
// l / 16 and l / 16 + 4 of its row's 128-byte line, and LDS is laid out as in gemm.hip (whole
// lines, XOR-swizzled chunks).
//
// The operands are swapped (B is the first), so a lane's four results are four consecutive n
// of one m: its scale of A is one value, and C is stored in 16-byte pieces.
//
// Scales.  e8m0 bytes go into the 8-bit instruction, or into the widening, and the products
// accumulate in place.  fp32 scales cannot: the block's product starts from zero and one fma per
// result folds it into the accumulator with sa sb; with a 128 x 128 scale of B that factor is
// one value per 16 rows for the whole wave, with one scale per row of B a vector of four.
// A stage's scales are staged in LDS beside its operands: thread t of the workgroup (as many
// threads as rows of A and B) loads entry t.

namespace engram {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

struct GemmFp8KArgs {
  const uint8_t* A;
  const uint8_t* B;
  const void* sa;
  const void* sb;
  void* C;
  int64_t lda, ldb, ldc, c_split_stride;
  int32_t M, N, KB;
  int32_t sb_ld, b_shift;    // entries per k block of sb; 0 or 7: row n reads entry n >> b_shift
  int32_t tiles_m, tiles_n, group_m;
  int32_t kb_per_split;
  int32_t c_f32, vec_store;
};

// A barrier that the compiler moves no memory access across (the builtin alone only stops
// the hardware); the waits that make LDS contents visible are the caller's.
__device__ __forceinline__ void stage_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// 32 codes to bf16, times 2^(byte - 127): the operands of four k32 steps
__device__ __forceinline__ void widen_codes(const i32x8& q, float scale, bf16x8* o) {
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    bf16x2 p[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      p[2 * h] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)q[2 * s + h], scale, false);
      p[2 * h + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)q[2 * s + h], scale, true);
    }
    o[s] = bf16x8{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
  }
}

template <int BM, int BN, int WM_WAVES, int WN_WAVES, bool WIDE, bool E8M0, bool B_ROWS>
__device__ __forceinline__ void gemm_fp8_tile(const GemmFp8KArgs& a) {
  constexpr int NWAVES = WM_WAVES * WN_WAVES, THREADS = NWAVES * 64;
  constexpr int WM = BM / WM_WAVES, WN = BN / WN_WAVES, TM = WM / 16, TN = WN / 16;
  constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  constexpr int SCALES = A_BYTES + B_BYTES;               // byte offset of the scales in a stage
  constexpr int STAGE = SCALES + (BM + BN) * 4;
  constexpr int AI = BM / 8 / NWAVES, BI = BN / 8 / NWAVES;  // 1 KB direct loads per wave and stage
  static_assert(BM + BN == THREADS, "one scale per thread and stage");
  static_assert(128 % WN == 0, "a wave's columns share their 128-block");
  extern __shared__ __attribute__((aligned(1024))) char smem[];

  const int ntiles = a.tiles_m * a.tiles_n;
  int bid = blockIdx.x;
  const int split = bid / ntiles;
  bid -= split * ntiles;
  if ((ntiles & 7) == 0) {
    const int per_xcd = ntiles >> 3;
    bid = (bid & 7) * per_xcd + (bid >> 3);
  }
  const int group = a.group_m * a.tiles_n;
  const int gid = bid / group;
  const int first_m = gid * a.group_m;
  const int gm = min(a.tiles_m - first_m, a.group_m);
  const int in_group = bid - gid * group;
  const int m0 = (first_m + in_group % gm) * BM;
  const int n0 = (in_group / gm) * BN;
  const int kb0 = split * a.kb_per_split;
  const int nk = min(a.kb_per_split, a.KB - kb0);

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WN_WAVES, wn = wave % WN_WAVES;
  const int rows_a = min(a.M - m0, BM), rows_b = min(a.N - n0, BN);
  const __amdgpu_buffer_rsrc_t arsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(a.A + (int64_t)m0 * a.lda), (short)0, (int)((int64_t)rows_a * a.lda), kBufferRsrcFlags);
  const __amdgpu_buffer_rsrc_t brsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(a.B + (int64_t)n0 * a.ldb), (short)0, (int)((int64_t)rows_b * a.ldb), kBufferRsrcFlags);

  // direct loads: wave w, load i fills LDS bytes [(NWAVES i + w) KB, +1 KB) of the operand;
  // 8 lanes fetch one row's 128 bytes.  Rows past the matrix read its last row (never stored).
  int aoff[AI], boff[BI];
#pragma unroll
  for (int i = 0; i < AI; ++i) {
    const int P = 64 * (i * NWAVES + wave) + lane, row = P >> 3, c = (P & 7) ^ gemm_swz(row);
    aoff[i] = min(row, rows_a - 1) * (int)a.lda + 16 * c;
  }
#pragma unroll
  for (int i = 0; i < BI; ++i) {
    const int P = 64 * (i * NWAVES + wave) + lane, row = P >> 3, c = (P & 7) ^ gemm_swz(row);
    boff[i] = min(row, rows_b - 1) * (int)a.ldb + 16 * c;
  }
  auto issue = [&](int kt) {
    char* st = smem + (kt & 1) * STAGE;
    const int k = (kb0 + kt) * 128;
#pragma unroll
    for (int i = 0; i < AI; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(arsrc, (ENGRAM_LDS_AS void*)(st + (i * NWAVES + wave) * 1024), 16,
                                               aoff[i] + k, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < BI; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(brsrc, (ENGRAM_LDS_AS void*)(st + A_BYTES + (i * NWAVES + wave) * 1024),
                                               16, boff[i] + k, 0, 0, 0);
  };
  // the thread's scale entry: rows of A first, then rows (or 128-blocks) of B
  const bool is_a = tid < BM;
  const int64_t s_ld = is_a ? a.M : a.sb_ld;
  const int64_t s_at = is_a ? m0 + min(tid, rows_a - 1) : (n0 + min(tid - BM, rows_b - 1)) >> a.b_shift;
  const void* s_base = is_a ? a.sa : a.sb;
  auto load_scale = [&](int kt) -> uint32_t {
    const int64_t e = (int64_t)(kb0 + kt) * s_ld + s_at;
    return E8M0 ? (uint32_t) static_cast<const uint8_t*>(s_base)[e] : static_cast<const uint32_t*>(s_base)[e];
  };
  auto put_scale = [&](int kt, uint32_t s) {
    reinterpret_cast<uint32_t*>(smem + (kt & 1) * STAGE + SCALES)[tid] = s;
  };

  const int lrow = lane & 15, lk = lane >> 4;
  auto fragment = [&](const char* base, int row) -> i32x8 {
    const char* p = base + row * 128;
    const int z = gemm_swz(row);
    const i32x4 lo = *reinterpret_cast<const i32x4*>(p + 16 * (lk ^ z));
    const i32x4 hi = *reinterpret_cast<const i32x4*>(p + 16 * ((lk + 4) ^ z));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };

  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{};

  uint32_t sreg = load_scale(0);
  issue(0);
  wait_vmcnt<0>();
  put_scale(0, sreg);
  wait_lgkmcnt0();
  stage_barrier();
  for (int kt = 0; kt < nk; ++kt) {
    const bool more = kt + 1 < nk;
    if (more) {
      sreg = load_scale(kt + 1);
      issue(kt + 1);
    }
    const char* st = smem + (kt & 1) * STAGE;
    const uint32_t* sc = reinterpret_cast<const uint32_t*>(st + SCALES);
    const uint32_t* sca = sc + wm * WM + lrow;
    const uint32_t* scb = sc + BM + wn * WN;
    // The columns' fragments stay in registers for the stage; the rows' are fetched one 16-row
    // tile ahead of the products.  The scheduling barriers keep the compiler from fetching
    // every tile at once, which spills.
    i32x8 fb[WIDE ? 1 : TN];
    bf16x8 wb[WIDE ? TN : 1][4];
    uint32_t sb1[TN];
    f32x4 sb4[TN];
    i32x8 fa = fragment(st, wm * WM + lrow);
    uint32_t sa = sca[0];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const i32x8 f = fragment(st + A_BYTES, wn * WN + j * 16 + lrow);
      if (E8M0) sb1[j] = scb[j * 16 + lrow];
      else if (B_ROWS) sb4[j] = *reinterpret_cast<const f32x4*>(scb + j * 16 + 4 * lk);
      if (WIDE) widen_codes(f, E8M0 ? e8m0_value(sb1[j]) : 1.0f, wb[j]);
      else fb[j] = f;
    }
    const float sbw = !E8M0 && !B_ROWS ? __uint_as_float(scb[0]) : 1.0f;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      bf16x8 wa[4];
      if (WIDE) widen_codes(fa, E8M0 ? e8m0_value(sa) : 1.0f, wa);
      const i32x8 f = fa;
      const uint32_t s1 = sa;
      if (i + 1 < TM) {
        fa = fragment(st, wm * WM + (i + 1) * 16 + lrow);
        sa = sca[(i + 1) * 16];
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        if (E8M0) {
          if (WIDE) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j][q], wa[q], acc[i][j], 0, 0, 0);
          } else {
            acc[i][j] =
                __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], f, acc[i][j], 0, 0, 0, (int)sb1[j], 0, (int)s1);
          }
        } else {
          f32x4 p = {};
          if (WIDE) {
#pragma unroll
            for (int q = 0; q < 4; ++q) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j][q], wa[q], p, 0, 0, 0);
          } else {
            p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], f, p, 0, 0, 0, 0, 0, 0);
          }
          const float s = __uint_as_float(s1) * sbw;
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[i][j][v] = fmaf(p[v], B_ROWS ? __uint_as_float(s1) * sb4[j][v] : s, acc[i][j][v]);
          // keeps the fold here: moved behind all products, as the compiler would, it holds
          // every product's registers at once
          asm volatile("" : "+v"(acc[i][j]));
        }
      }
    }
    if (more) {
      wait_vmcnt<0>();
      put_scale(kt + 1, sreg);
    }
    wait_lgkmcnt0();
    stage_barrier();
  }

  // lane: row m = lrow, columns 4 lk .. +4 of each 16 x 16 tile
  const int64_t base = (int64_t)split * a.c_split_stride;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int m = m0 + wm * WM + i * 16 + lrow;
    if (m >= a.M) continue;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int n = n0 + wn * WN + j * 16 + 4 * lk;
      if (n >= a.N) continue;
      const int64_t at = base + (int64_t)m * a.ldc + n;
      if (a.vec_store && n + 4 <= a.N) {
        if (a.c_f32) {
          *reinterpret_cast<f32x4*>(static_cast<float*>(a.C) + at) = acc[i][j];
        } else {
          uint2 o;
          o.x = bf16_bits_rne(acc[i][j][0]) | (bf16_bits_rne(acc[i][j][1]) << 16);
          o.y = bf16_bits_rne(acc[i][j][2]) | (bf16_bits_rne(acc[i][j][3]) << 16);
          *reinterpret_cast<uint2*>(static_cast<unsigned short*>(a.C) + at) = o;
        }
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (n + v < a.N) {
            if (a.c_f32) static_cast<float*>(a.C)[at + v] = acc[i][j][v];
            else static_cast<unsigned short*>(a.C)[at + v] = (unsigned short)bf16_bits_rne(acc[i][j][v]);
          }
      }
    }
  }
}

template <int BM, int BN, int WM_WAVES, int WN_WAVES, bool WIDE, bool E8M0, bool B_ROWS>
__global__ __launch_bounds__(WM_WAVES* WN_WAVES * 64) void gemm_fp8_kernel(GemmFp8KArgs a) {
  gemm_fp8_tile<BM, BN, WM_WAVES, WN_WAVES, WIDE, E8M0, B_ROWS>(a);
}

// C = the sum of the split-K slices, in slice order
__global__ __launch_bounds__(256) void gemm_fp8_join_kernel(const float* __restrict__ work, int32_t splits, int64_t MN,
                                                            int32_t N, void* C, int32_t c_f32, int64_t ldc) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= MN) return;
  float s = work[i];
  for (int p = 1; p < splits; ++p) s += work[(int64_t)p * MN + i];
  const int64_t m = i / N, n = i - m * N;
  if (c_f32) static_cast<float*>(C)[m * ldc + n] = s;
  else static_cast<unsigned short*>(C)[m * ldc + n] = (unsigned short)bf16_bits_rne(s);
}

struct GemmFp8Plan {
  int bm, splits;
};

static GemmFp8Plan gemm_fp8_plan(int64_t M, int64_t N, int64_t KB) {
  GemmFp8Plan p = {256, 1};
  const int64_t big = ((M + 255) / 256) * ((N + 255) / 256);
  if (big >= 192) return p;
  p.bm = 128;
  const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);
  while (tiles * p.splits * 2 <= 256 && KB / (p.splits * 2) >= 2) p.splits *= 2;
  return p;
}

int64_t gemm_fp8_workspace_bytes(int64_t M, int64_t N, int64_t KB) {
  const GemmFp8Plan p = gemm_fp8_plan(M, N, KB);
  return p.splits > 1 ? (int64_t)p.splits * M * N * 4 : 0;
}

template <int BM, int WM_WAVES, int WN_WAVES, bool WIDE, bool E8M0, bool B_ROWS>
static hipError_t gemm_fp8_start(const GemmFp8KArgs& a, int64_t grid, hipStream_t stream) {
  constexpr int lds = 2 * (BM * 256 + BM * 8);
  static std::atomic<uint64_t> lds_set{0};
  const hipError_t e = ensure_dynamic_lds(
      reinterpret_cast<const void*>(&gemm_fp8_kernel<BM, BM, WM_WAVES, WN_WAVES, WIDE, E8M0, B_ROWS>), lds, lds_set);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((gemm_fp8_kernel<BM, BM, WM_WAVES, WN_WAVES, WIDE, E8M0, B_ROWS>), dim3((unsigned)grid),
                     dim3(WM_WAVES * WN_WAVES * 64), lds, stream, a);
  return hipGetLastError();
}

template <int BM, int WM_WAVES, int WN_WAVES, bool WIDE>
static hipError_t gemm_fp8_kinds(const GemmFp8Args& g, const GemmFp8KArgs& a, int64_t grid, hipStream_t stream) {
  if (g.e8m0) return gemm_fp8_start<BM, WM_WAVES, WN_WAVES, WIDE, true, false>(a, grid, stream);
  if (g.b_block == 1) return gemm_fp8_start<BM, WM_WAVES, WN_WAVES, WIDE, false, true>(a, grid, stream);
  return gemm_fp8_start<BM, WM_WAVES, WN_WAVES, WIDE, false, false>(a, grid, stream);
}

hipError_t launch_gemm_fp8(const GemmFp8Args& g, hipStream_t stream) {
  (void)hipGetLastError();
  if (g.M == 0 || g.N == 0) return hipSuccess;
  const GemmFp8Plan p = gemm_fp8_plan(g.M, g.N, g.KB);
  GemmFp8KArgs a;
  a.A = g.A;
  a.B = g.B;
  a.sa = g.sa;
  a.sb = g.sb;
  a.lda = g.lda;
  a.ldb = g.ldb;
  a.M = g.M;
  a.N = g.N;
  a.KB = g.KB;
  a.sb_ld = g.b_block == 1 ? g.N : (g.N + 127) / 128;
  a.b_shift = g.b_block == 1 ? 0 : 7;
  a.tiles_m = (g.M + p.bm - 1) / p.bm;
  a.tiles_n = (g.N + p.bm - 1) / p.bm;
  a.group_m = 4;
  a.kb_per_split = (g.KB + p.splits - 1) / p.splits;
  const int splits = (g.KB + a.kb_per_split - 1) / a.kb_per_split;  // every split has work
  const bool joined = splits > 1;
  a.C = joined ? (void*)g.work : g.C;
  a.c_f32 = joined ? 1 : g.c_f32;
  a.ldc = joined ? g.N : g.ldc;
  a.c_split_stride = joined ? (int64_t)g.M * g.N : 0;
  a.vec_store = (a.ldc % 4 == 0 && a.c_split_stride % 4 == 0 && ((uintptr_t)a.C & 15) == 0) ? 1 : 0;
  const int64_t grid = (int64_t)a.tiles_m * a.tiles_n * splits;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipError_t e;
  if (p.bm == 256)
    e = g.c_f32 ? gemm_fp8_kinds<256, 2, 4, true>(g, a, grid, stream) : gemm_fp8_kinds<256, 2, 4, false>(g, a, grid, stream);
  else
    e = g.c_f32 ? gemm_fp8_kinds<128, 2, 2, true>(g, a, grid, stream) : gemm_fp8_kinds<128, 2, 2, false>(g, a, grid, stream);
  if (e != hipSuccess || !joined) return e;
  const int64_t MN = (int64_t)g.M * g.N;
  hipLaunchKernelGGL(gemm_fp8_join_kernel, dim3((unsigned)((MN + 255) / 256)), dim3(256), 0, stream, g.work, splits, MN,
                     g.N, g.C, g.c_f32, g.ldc);
  return hipGetLastError();
}

}  // namespace engram
