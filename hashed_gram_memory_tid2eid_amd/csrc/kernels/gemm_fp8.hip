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
// - fp32 C: the codes are widened to bf16 in registers, exactly (with an e8m0 scale from 2^-124
//   on: a code's last bit is 2^-9, bf16's 2^-133), and multiplied by
//   v_mfma_f32_16x16x32_bf16, whose sums keep fp32 (1e-7 at K = 6,144), at half the rate.
//   The 8-bit instruction of that shape (16x16x32) has this rate and the short sums.
//
// A lane's operand is 32 codes of one row; which 32 of the block's 128 does not matter as
// long as both operands agree (the scale is one for all 128), so a lane takes 16-byte chunks
// l / 16 and l / 16 + 4 of its row's 128-byte line, and LDS is laid out as in gemm.hip (whole
// lines, XOR-swizzled chunks).
//
// The operands are swapped (B is the first), so a lane's four results are four consecutive n
// of one m, and its scale of A is one value.
//
// Scales.  e8m0 bytes go into the 8-bit instruction, or into the widening, and the products
// accumulate in place.  fp32 scales cannot: the block's product starts from zero and one fma per
// result folds it into the accumulator with sa sb; with a 128 x 128 scale of B that factor is
// one value per lane and row tile, with one scale per row of B a vector of four.
// A stage's scales are staged in LDS beside its operands: thread t of the workgroup (as many
// threads as rows of A and B) loads entry t.
//
// What bounds it is the issue of a SIMD, which the matrix and the vector instructions share:
// about 4.7 cycles times their number.  65,536 x 4,096 over 6,144 (3.3e12 operations), medians of 40
// calls, least 2 to 4% lower: bf16 C with e8m0 scales 1,303 us (2.53 PFLOP/s), fp32 1,487 us (2.22),
// fp32 with one per row of B 1,697 us (1.94); fp32 C 2,268 us (1.45), 2,431 us (1.36) and 2,863 us
// (1.15): the widening is a vector instruction per 4 codes, an fp32 scale an fma per result and
// block more.
// Measured and not taken: 32 x 32 matrix shapes (the same; e8m0 15% slower), 4 waves of 128 x 128
// (the accumulators leave the vector registers, and the folds pay the moves), B widened during
// the last row tile before the barrier (spills), a branch between full and edge tiles around the
// loads (15% slower: they can no longer be spread over the stage), waves that alternate between
// vector and matrix phases by priority (the same).

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
  int64_t lda, ldb, ldc;
  int32_t M, N, KB;
  int32_t sb_ld, b_shift;    // entries per k block of sb; 0 or 7: row n reads entry n >> b_shift
  int32_t tiles_m, tiles_n, group_m;
  int32_t whole;             // tiles 0 .. whole - 1 run over all of K; the others in splits of it
  int32_t kb_per_split;
  float* work;               // the splits' tiles: [split][tile - whole][BM][BN]
  int32_t c_f32, vec_store;
};

// What a workgroup computes: a tile over all of K, or one split of a tile (part: which of the
// splits' tiles in the workspace; -1: none, the tile goes to C).
struct GemmFp8Tile {
  int m, n, split, part;
};

__device__ __forceinline__ GemmFp8Tile gemm_fp8_tile_of(const GemmFp8KArgs& a, int block) {
  GemmFp8Tile o = {0, 0, 0, -1};
  int tile = block;
  if (block >= a.whole) {
    const int rest = a.tiles_m * a.tiles_n - a.whole;
    o.part = block - a.whole;
    o.split = o.part / rest;
    tile = a.whole + (o.part - o.split * rest);
  } else if ((a.whole & 7) == 0) {  // each XCD takes a run of consecutive tiles
    tile = (block & 7) * (a.whole >> 3) + (block >> 3);
  }
  const int group = a.group_m * a.tiles_n;
  const int gid = tile / group;
  const int first_m = gid * a.group_m;
  const int gm = min(a.tiles_m - first_m, a.group_m);
  const int in_group = tile - gid * group;
  o.m = first_m + in_group % gm;
  o.n = in_group / gm;
  return o;
}

// A barrier that the compiler moves no memory access across (the builtin alone only stops
// the hardware); the waits that make LDS contents visible are the caller's.
__device__ __forceinline__ void stage_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// 32 codes to bf16, times a power of two: the operands of four k32 steps
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

  const GemmFp8Tile at = gemm_fp8_tile_of(a, blockIdx.x);
  const int m0 = at.m * BM, n0 = at.n * BN;
  const int kb0 = at.split * a.kb_per_split;
  const int nk = at.part < 0 ? a.KB : min(a.kb_per_split, a.KB - kb0);

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN_WAVES, wn = wave % WN_WAVES;
  const int rows_a = min(a.M - m0, BM), rows_b = min(a.N - n0, BN);
  const __amdgpu_buffer_rsrc_t arsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(a.A + (int64_t)m0 * a.lda), (short)0, (int)((int64_t)rows_a * a.lda), kBufferRsrcFlags);
  const __amdgpu_buffer_rsrc_t brsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(a.B + (int64_t)n0 * a.ldb), (short)0, (int)((int64_t)rows_b * a.ldb), kBufferRsrcFlags);

  // direct loads: wave w, load i fills LDS bytes [(NWAVES i + w) KB, +1 KB) of the operand;
  // 8 lanes fetch one row's 128 bytes.  Rows past the matrix read its last row (never stored).
  int offset[AI + BI];
#pragma unroll
  for (int i = 0; i < AI + BI; ++i) {
    const bool of_a = i < AI;
    const int row = ((of_a ? i : i - AI) * NWAVES + wave) * 8 + (lane >> 3), c = (lane & 7) ^ gemm_swz(row);
    offset[i] = min(row, (of_a ? rows_a : rows_b) - 1) * (int)(of_a ? a.lda : a.ldb) + 16 * c;
  }
  // load i of stage kt; stages past the end: the last one again, into a slot nobody reads
  auto issue = [&](int kt, int i) {
    const int k = (kb0 + min(kt, nk - 1)) * 128;
    const int to = (kt & 1) * STAGE + (i < AI ? i : i - AI) * NWAVES * 1024 + (i < AI ? 0 : A_BYTES) + wave * 1024;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(i < AI ? arsrc : brsrc, (ENGRAM_LDS_AS void*)(smem + to), 16, offset[i], k, 0,
                                             0);
  };
  // the thread's scale entry: rows of A first, then rows (or 128-blocks) of B
  const bool is_a = wave * 64 < BM;
  const int64_t s_ld = is_a ? a.M : a.sb_ld;
  const char* s_base = static_cast<const char*>(is_a ? a.sa : a.sb) + (int64_t)kb0 * s_ld * (E8M0 ? 1 : 4);
  const int s_at = is_a ? m0 + min(tid, rows_a - 1) : (n0 + min(tid - BM, rows_b - 1)) >> a.b_shift;
  auto load_scale = [&](int kt) -> uint32_t {
    const char* p = s_base + min(kt, nk - 1) * s_ld * (E8M0 ? 1 : 4);
    return E8M0 ? (uint32_t)reinterpret_cast<const uint8_t*>(p)[s_at] : reinterpret_cast<const uint32_t*>(p)[s_at];
  };
  auto put_scale = [&](int kt, uint32_t s) {
    reinterpret_cast<uint32_t*>(smem + (kt & 1) * STAGE + SCALES)[tid] = s;
  };

  const int lrow = lane & 15, lk = lane >> 4;
  // row r0 + l % 16's codes (r0 a multiple of 16, whose rows share the swizzle)
  const int off0 = lrow * 128 + 16 * (lk ^ gemm_swz(lrow)), off1 = lrow * 128 + 16 * ((lk + 4) ^ gemm_swz(lrow));
  auto fragment = [&](const char* base, int r0) -> i32x8 {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(base + r0 * 128 + off0);
    const i32x4 hi = *reinterpret_cast<const i32x4*>(base + r0 * 128 + off1);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };

  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{};

  // fp32 scales: the block product of the tile before the current one, still to be folded
  // into its accumulator (times its scales) while the current one multiplies
  f32x4 p_old = {}, s_old = {};
  auto fold = [&](int i, int j) {
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(p_old[v], B_ROWS ? s_old[v] : s_old[0], acc[i][j][v]);
    // keeps the fold here: moved behind all products, as the compiler would, it holds every
    // product's registers at once
    asm volatile("" : "+v"(acc[i][j]));
  };

  uint32_t sreg = load_scale(0);
#pragma unroll
  for (int i = 0; i < AI + BI; ++i) issue(0, i);
  wait_vmcnt<0>();
  put_scale(0, sreg);
  wait_lgkmcnt0();
  stage_barrier();
  for (int kt = 0; kt < nk; ++kt) {
    // past the end: the last stage again, into a slot nobody reads
    sreg = load_scale(kt + 1);
    const char* st = smem + (kt & 1) * STAGE;
    const char* sta = st + wm * WM * 128;
    const char* stb = st + A_BYTES + wn * WN * 128;
    const uint32_t* sca = reinterpret_cast<const uint32_t*>(st + SCALES) + wm * WM + lrow;
    const uint32_t* scb = reinterpret_cast<const uint32_t*>(st + SCALES) + BM + wn * WN;
    i32x8 fb[TN];
    bf16x8 wb[WIDE ? TN : 1][4];
    uint32_t sb1[TN];
    f32x4 sb4[TN];  // one scale per row of B: held for the stage, or (WIDE, no registers) read where used
    auto fetch_b = [&](int j) {
      fb[j] = fragment(stb, j * 16);
      if (E8M0) sb1[j] = scb[j * 16 + lrow];
      if (!E8M0 && B_ROWS && !WIDE) sb4[j] = *reinterpret_cast<const f32x4*>(scb + j * 16 + 4 * lk);
    };
    fetch_b(0);
    i32x8 fa = fragment(sta, 0);
    uint32_t sa = sca[0];
    const float sbw = !E8M0 && !B_ROWS ? __uint_as_float(scb[0]) : 1.0f;
    if (TN > 1) fetch_b(1);
    if (WIDE) widen_codes(fb[0], E8M0 ? e8m0_value(sb1[0]) : 1.0f, wb[0]);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      // Of the two waves of a SIMD the one that is behind goes first: left to their age, the
      // older four run ahead, wait at the barrier for a third of the stage, and each wave
      // alone cannot keep the matrix cores fed.  (Tiles of 128 run two or three workgroups
      // per CU, and were up to 15% slower with it.)
      if (BM == 256 && i % (TM / 4) == 0) {
        if (i * 4 / TM == 0) __builtin_amdgcn_s_setprio(3);
        if (i * 4 / TM == 1) __builtin_amdgcn_s_setprio(2);
        if (i * 4 / TM == 2) __builtin_amdgcn_s_setprio(1);
        if (i * 4 / TM == 3) __builtin_amdgcn_s_setprio(0);
      }
      // the next stage's loads, spread over the first row tiles: issued at once they held the
      // wave for up to a thousand of a stage's 5,000 to 8,000 cycles
      constexpr int PER = (AI + BI + TM / 2 - 1) / (TM / 2);
#pragma unroll
      for (int e = 0; e < PER; ++e)
        if (i * PER + e < AI + BI) issue(kt + 1, i * PER + e);
      bf16x8 wa[4];
      if (WIDE) widen_codes(fa, E8M0 ? e8m0_value(sa) : 1.0f, wa);
      const i32x8 f = fa;
      const uint32_t s1 = sa;
      if (i + 1 < TM) {  // the next row tile, one ahead of the products
        fa = fragment(sta, (i + 1) * 16);
        sa = sca[(i + 1) * 16];
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        // one tile: its products, the fold of the tile before, and in the first row tile the
        // next columns' operands.  Nothing crosses to another tile: free to, the compiler
        // fetches and folds everything at once, and spills.
        __builtin_amdgcn_sched_barrier(0);
        f32x4 p = E8M0 ? acc[i][j] : f32x4{};
        if (WIDE) {
#pragma unroll
          for (int q = 0; q < 4; ++q) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j][q], wa[q], p, 0, 0, 0);
        } else if (E8M0) {
          p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], f, p, 0, 0, 0, (int)sb1[j], 0, (int)s1);
        } else {
          p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], f, p, 0, 0, 0, 0, 0, 0);
        }
        if (i == 0 && j + 2 < TN) fetch_b(j + 2);
        if (WIDE && i == 0 && j + 1 < TN) widen_codes(fb[j + 1], E8M0 ? e8m0_value(sb1[j + 1]) : 1.0f, wb[j + 1]);
        if (E8M0) {
          acc[i][j] = p;
        } else {
          const int t = i * TN + j + TM * TN - 1;
          fold(t / TN % TM, t % TN);
          p_old = p;
          if (B_ROWS && WIDE) sb4[j] = *reinterpret_cast<const f32x4*>(scb + j * 16 + 4 * lk);
          if (B_ROWS) s_old = __uint_as_float(s1) * sb4[j];
          else s_old[0] = __uint_as_float(s1) * sbw;
        }
      }
    }
    wait_vmcnt<0>();
    put_scale(kt + 1, sreg);
    wait_lgkmcnt0();
    stage_barrier();
  }
  if (!E8M0) fold(TM - 1, TN - 1);

  // C: lane l holds of each 16 x 16 tile row m = l % 16 and columns 4 (l / 16) .. +4.
  // Each wave lays 16 rows of its columns out in LDS (the ring is done with: the loads of the
  // stage past the end have landed) and writes them as whole row segments.
  constexpr int PITCH = WN + 4;
  static_assert(NWAVES * 16 * PITCH * 4 <= 2 * STAGE, "the slabs fit in the ring");
  float* slab = reinterpret_cast<float*>(smem) + wave * 16 * PITCH;
  // the tile in C, or the split's in the workspace; where it is is worked out again, so that
  // the loop need not hold it
  int block = blockIdx.x;
  asm volatile("" : "+s"(block));
  const GemmFp8Tile to = gemm_fp8_tile_of(a, block);
  const bool part = to.part >= 0;
  void* const out = part ? (void*)(a.work + (int64_t)to.part * (BM * BN))
                         : (void*)(static_cast<char*>(a.C) + ((int64_t)to.m * BM * a.ldc + to.n * BN) * (a.c_f32 ? 4 : 2));
  const int left_m = a.M - to.m * BM, left_n = a.N - to.n * BN;
  const int64_t ld = part ? BN : a.ldc;
  const bool out_f32 = part || a.c_f32, vec = part || a.vec_store;
  constexpr int LANES = WN / 4, ROWS = 64 / LANES;  // lanes per row, rows per pass
  const int n = wn * WN + (lane % LANES) * 4;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j) *reinterpret_cast<f32x4*>(slab + lrow * PITCH + j * 16 + 4 * lk) = acc[i][j];
    asm volatile("" ::: "memory");  // a wave's own LDS accesses keep their order
#pragma unroll
    for (int q = 0; q < 16 / ROWS; ++q) {
      const int r = q * ROWS + lane / LANES;
      const f32x4 val = *reinterpret_cast<const f32x4*>(slab + r * PITCH + (lane % LANES) * 4);
      const int m = wm * WM + i * 16 + r;
      if (m >= left_m || n >= left_n) continue;
      const int64_t at = (int64_t)m * ld + n;
      if (vec && n + 4 <= left_n) {
        if (out_f32) {
          *reinterpret_cast<f32x4*>(static_cast<float*>(out) + at) = val;
        } else {
          uint2 o;
          o.x = bf16_bits_rne(val[0]) | (bf16_bits_rne(val[1]) << 16);
          o.y = bf16_bits_rne(val[2]) | (bf16_bits_rne(val[3]) << 16);
          *reinterpret_cast<uint2*>(static_cast<unsigned short*>(out) + at) = o;
        }
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (n + v < left_n) {
            if (out_f32) static_cast<float*>(out)[at + v] = val[v];
            else static_cast<unsigned short*>(out)[at + v] = (unsigned short)bf16_bits_rne(val[v]);
          }
      }
    }
    asm volatile("" ::: "memory");
  }
}

template <int BM, int BN, int WM_WAVES, int WN_WAVES, bool WIDE, bool E8M0, bool B_ROWS>
__global__ __launch_bounds__(WM_WAVES* WN_WAVES * 64) void gemm_fp8_kernel(GemmFp8KArgs a) {
  gemm_fp8_tile<BM, BN, WM_WAVES, WN_WAVES, WIDE, E8M0, B_ROWS>(a);
}

// The tiles whose K was split: C = the sum of their splits, in order.  A workgroup joins 1,024
// elements of one tile, 4 a thread.
template <int BM>
__global__ __launch_bounds__(256) void gemm_fp8_join_kernel(GemmFp8KArgs a, int32_t splits) {
  constexpr int PER = BM * BM / 1024;
  const int rest = a.tiles_m * a.tiles_n - a.whole;
  const int t = blockIdx.x / PER, e = (blockIdx.x % PER) * 1024 + threadIdx.x * 4;
  const GemmFp8Tile tile = gemm_fp8_tile_of(a, a.whole + t);
  const int m = tile.m * BM + e / BM, n = tile.n * BM + e % BM;
  if (m >= a.M || n >= a.N) return;
  const float* w = a.work + (int64_t)t * (BM * BM) + e;
  f32x4 s = *reinterpret_cast<const f32x4*>(w);
  for (int p = 1; p < splits; ++p) s += *reinterpret_cast<const f32x4*>(w + (int64_t)p * rest * (BM * BM));
  const int64_t at = (int64_t)m * a.ldc + n;
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (n + v < a.N) {
      if (a.c_f32) static_cast<float*>(a.C)[at + v] = s[v];
      else static_cast<unsigned short*>(a.C)[at + v] = (unsigned short)bf16_bits_rne(s[v]);
    }
}

// ---- few rows of A ----------------------------------------------------------------
//
// Up to 16 MT rows (MT 1 or 2): the weight's bytes are the work, and what counts is how many of them are
// on their way.  One workgroup owns 16 columns and all of K, its 16 waves every 16th k block
// of them, straight from memory into the operand registers (no LDS, no stages): 256
// workgroups hold 4,096 columns, each wave some 6 KB of weight in flight.  The waves' sums meet
// in LDS and are added in wave order; there is no second launch and no workspace.
// Weights from memory, 4,096 columns, K 6,144, in a replayed graph: 1 row 7.3 us, 16 rows 9.1, 32
// rows 12.2 (cached 6.3, 8.0, 11.0).  Called one by one from the host 16 and 32 rows took 11.4 and
// 14.8; with 8 waves of 4 blocks in flight 13.3 and 17.7, of 6 blocks 11.6 and 14.7 (but K 19,584 28
// against 25), with 16 waves of 2 blocks 11.8 and 14.6.  25 MB take 4 us of memory's rate.

constexpr int kFewWaves = 16;

template <int MT, bool WIDE, bool E8M0, bool B_ROWS>
__device__ __forceinline__ void gemm_fp8_few_rows(const GemmFp8KArgs& a) {
  constexpr int U = 3;  // k blocks in flight
  __shared__ f32x4 part[kFewWaves][MT][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lrow = lane & 15, lk = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int nb = min(n0 + lrow, a.N - 1);
  const uint8_t* b = a.B + (int64_t)nb * a.ldb + 16 * lk;
  const uint8_t* ap[MT];
  int ma[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    ma[i] = min(i * 16 + lrow, a.M - 1);
    ap[i] = a.A + (int64_t)ma[i] * a.lda + 16 * lk;
  }
  auto scale_at = [&](const void* base, int64_t at) -> uint32_t {
    return E8M0 ? (uint32_t) static_cast<const uint8_t*>(base)[at] : static_cast<const uint32_t*>(base)[at];
  };
  auto codes = [](const uint8_t* p) -> i32x8 {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(p), hi = *reinterpret_cast<const i32x4*>(p + 64);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{};
  for (int k0 = wave; k0 < a.KB; k0 += kFewWaves * U) {
    i32x8 fb[U], fa[U][MT];
    uint32_t sb[U][4], sa[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = min(k0 + u * kFewWaves, a.KB - 1);  // past the end: loaded, not used
      fb[u] = codes(b + (int64_t)kb * 128);
      if (E8M0) {
        sb[u][0] = scale_at(a.sb, (int64_t)kb * a.sb_ld + (nb >> a.b_shift));
      } else {
#pragma unroll
        for (int v = 0; v < (B_ROWS ? 4 : 1); ++v)
          sb[u][v] = scale_at(a.sb, (int64_t)kb * a.sb_ld + (min(n0 + 4 * lk + v, a.N - 1) >> a.b_shift));
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        fa[u][i] = codes(ap[i] + (int64_t)kb * 128);
        sa[u][i] = scale_at(a.sa, (int64_t)kb * a.M + ma[i]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u * kFewWaves >= a.KB) continue;  // uniform
      bf16x8 wb[4], wa[4];
      if (WIDE) widen_codes(fb[u], E8M0 ? e8m0_value(sb[u][0]) : 1.0f, wb);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if (WIDE) widen_codes(fa[u][i], E8M0 ? e8m0_value(sa[u][i]) : 1.0f, wa);
        f32x4 p = E8M0 ? acc[i] : f32x4{};
        if (WIDE) {
#pragma unroll
          for (int q = 0; q < 4; ++q) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[q], wa[q], p, 0, 0, 0);
        } else if (E8M0) {
          p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[u], fa[u][i], p, 0, 0, 0, (int)sb[u][0], 0, (int)sa[u][i]);
        } else {
          p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[u], fa[u][i], p, 0, 0, 0, 0, 0, 0);
        }
        if (E8M0) {
          acc[i] = p;
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[i][v] = fmaf(p[v], __uint_as_float(sa[u][i]) * __uint_as_float(sb[u][B_ROWS ? v : 0]), acc[i][v]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  for (int t = tid; t < MT * 64; t += kFewWaves * 64) {
    const int i = t >> 6, l = t & 63;
    f32x4 s = part[0][i][l];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) s += part[w][i][l];
    const int m = i * 16 + (l & 15), n = n0 + 4 * (l >> 4);
    if (m >= a.M) continue;
    const int64_t at = (int64_t)m * a.ldc + n;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (n + v < a.N) {
        if (a.c_f32) static_cast<float*>(a.C)[at + v] = s[v];
        else static_cast<unsigned short*>(a.C)[at + v] = (unsigned short)bf16_bits_rne(s[v]);
      }
  }
}

template <int MT, bool WIDE, bool E8M0, bool B_ROWS>
__global__ __launch_bounds__(kFewWaves * 64) void gemm_fp8_few_kernel(GemmFp8KArgs a) {
  gemm_fp8_few_rows<MT, WIDE, E8M0, B_ROWS>(a);
}

template <int MT, bool WIDE>
static void gemm_fp8_few_kinds(const GemmFp8Args& g, const GemmFp8KArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((g.N + 15) / 16)), block(kFewWaves * 64);
  if (g.e8m0) hipLaunchKernelGGL((gemm_fp8_few_kernel<MT, WIDE, true, false>), grid, block, 0, stream, a);
  else if (g.b_block == 1) hipLaunchKernelGGL((gemm_fp8_few_kernel<MT, WIDE, false, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((gemm_fp8_few_kernel<MT, WIDE, false, false>), grid, block, 0, stream, a);
}

template <bool WIDE>
static hipError_t gemm_fp8_few(const GemmFp8Args& g, const GemmFp8KArgs& a, hipStream_t stream) {
  if (g.M <= 16) gemm_fp8_few_kinds<1, WIDE>(g, a, stream);
  else gemm_fp8_few_kinds<2, WIDE>(g, a, stream);
  return hipGetLastError();
}

struct GemmFp8Plan {
  int bm;             // 256 or 128 (square tiles), 0: the few-row kernel
  int64_t whole;      // tiles that run over all of K
  int64_t rest;       // tiles whose K is split
  int splits;
};

// Up to this many rows the few-row kernel runs, which holds two row tiles.  4,096 columns, K 6,144,
// in a replayed graph, against 128 x 128 tiles with K split over 8 workgroups: weights from memory,
// 1 row 7.3 us against 17.2, 16 rows 9.1 against 18.7, 32 rows 12.2 against 19.6; cached 6.3 against
// 14.3, 8.0 against 16.3, 11.0 against 17.1.
constexpr int64_t kFewRows = 32;

// 256 x 256 tiles, one workgroup per CU, from 192 of them on; the tiles of a last, partly
// filled round are split over K, so that they fill it (4,096 x 6,144 over 16,384, 384 tiles:
// 656 -> 563 us with e8m0 scales).  Fewer tiles are 128 x 128, all of them split while there is a workgroup for
// every CU and two k blocks for each split.
static GemmFp8Plan gemm_fp8_plan(int64_t M, int64_t N, int64_t KB) {
  GemmFp8Plan p = {0, 0, 0, 1};
  if (M <= kFewRows) return p;
  int64_t tiles = ((M + 255) / 256) * ((N + 255) / 256);
  if (tiles >= 192) {
    p.bm = 256;
    p.rest = tiles > 256 ? tiles % 256 : 0;
    const int64_t s = p.rest > 0 ? 256 / p.rest : 1;
    // at least 8 k blocks to a split: a split's tile costs a write and a read of its sums
    p.splits = (int)(s < KB / 8 ? s : KB / 8);
    if (p.splits > 8) p.splits = 8;
  } else {
    p.bm = 128;
    tiles = ((M + 127) / 128) * ((N + 127) / 128);
    p.rest = tiles;
    while (tiles * p.splits * 2 <= 256 && KB / (p.splits * 2) >= 2) p.splits *= 2;
  }
  if (p.splits > 1) {  // every split has work
    const int64_t per = (KB + p.splits - 1) / p.splits;
    p.splits = (int)((KB + per - 1) / per);
  }
  if (p.splits <= 1) {
    p.splits = 1;
    p.rest = 0;
  }
  p.whole = tiles - p.rest;
  return p;
}

int64_t gemm_fp8_workspace_bytes(int64_t M, int64_t N, int64_t KB) {
  const GemmFp8Plan p = gemm_fp8_plan(M, N, KB);
  return p.rest * p.splits * p.bm * p.bm * 4;
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
  GemmFp8KArgs a = {};
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
  a.C = g.C;
  a.c_f32 = g.c_f32;
  a.ldc = g.ldc;
  if (p.bm == 0) return g.c_f32 ? gemm_fp8_few<true>(g, a, stream) : gemm_fp8_few<false>(g, a, stream);
  a.tiles_m = (g.M + p.bm - 1) / p.bm;
  a.tiles_n = (g.N + p.bm - 1) / p.bm;
  a.group_m = 4;
  a.whole = (int32_t)p.whole;
  a.kb_per_split = (g.KB + p.splits - 1) / p.splits;
  a.work = g.work;
  a.vec_store = (a.ldc % 4 == 0 && ((uintptr_t)a.C & 15) == 0) ? 1 : 0;
  const int64_t grid = p.whole + p.rest * p.splits;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipError_t e;
  if (p.bm == 256)
    e = g.c_f32 ? gemm_fp8_kinds<256, 2, 4, true>(g, a, grid, stream) : gemm_fp8_kinds<256, 2, 4, false>(g, a, grid, stream);
  else
    e = g.c_f32 ? gemm_fp8_kinds<128, 2, 2, true>(g, a, grid, stream) : gemm_fp8_kinds<128, 2, 2, false>(g, a, grid, stream);
  if (e != hipSuccess || p.rest == 0) return e;
  const int64_t joins = p.rest * (p.bm * p.bm / 1024);
  if (p.bm == 256)
    hipLaunchKernelGGL((gemm_fp8_join_kernel<256>), dim3((unsigned)joins), dim3(256), 0, stream, a, p.splits);
  else
    hipLaunchKernelGGL((gemm_fp8_join_kernel<128>), dim3((unsigned)joins), dim3(256), 0, stream, a, p.splits);
  return hipGetLastError();
}

}  // namespace engram
