// beam_select.hip -- beam search's selection over beams and vocabulary.  Included into
// engram_device.hip.
//
//   total(b, v) = score_b + x_bv - log sum_u exp(x_bu),  the n largest of a request's K * V
//
// Two launches.  The first cuts every row of logits into pieces of 256 lanes x NV loads of 16
// bytes, one workgroup each, and reads each logit once: a piece stays in registers while its
// maximum m is found, then its sum of exp(x - m) and its n largest logits.  Those need no sort
// of the piece: lane i of the four waves stands for the maximum of its elements (or each of the
// 256 threads for its own), and a bound that n of these maxima reach is reached by n elements at
// least and by few more.  The loads that hold such an element go to a list in LDS whole, the
// elements in them that reach the bound to a second one, and there each finds its rank by
// counting the larger ones.  Keys of (logit, lowest token first) are all different, so ranks
// are, too, whatever the order in which the lists were filled.  Long lists are not ranked: many
// logits are equal (masked by a finite number), or so near that the bound's 16 bits do not tell
// fp32 ones apart (a flat row).  The bound is then raised by bisection, counting in the registers,
// until few enough reach it or it is the n-th largest logit itself, whose equals follow those
// above it by their tokens.
// The second launch, one workgroup a request, adds the pieces' sums in 64 bits, turns the keys
// into totals and selects among them by the same bound, list and count, with the bound raised
// where many totals are nearly equal.
//
// Bound by memory where rows are many (2,048 x 129,280 fp32, 5% of them ended: 152 us, 7.0 TB/s in
// the first launch; bf16, 10% ended, 80 us, 6.0 TB/s), by latency below (4 rows 8.8 us, 512 rows
// of 65,537 bf16 22.2: their pieces all load, then all compute).  Where a mask's value or a flat row
// raises the bounds, the counts are on top: 2,048 x 129,280 masked by the lowest value, none
// ended, fp32 251 us, bf16 161 (161 and 91 without the mask).

namespace engram {

constexpr int kSelectThreads = 256;
constexpr int kSelectHeld = 4096;  // elements of the loads that hold one which reaches the bound
// Elements that reach it.  (Room past kSelectRanked leaves 5 workgroups of fp32 rows in a CU's LDS, which
// read faster than more of them.)
constexpr int kSelectList = 1024;
// Up to so many are ranked, each of which reads all.  64 candidates leave some 75, so that ordinary
// rows are below it (16 x 64 rows of 65,536 bf16, n 64: 41 us, 171 by 64; 4 flat rows of 129,280
// fp32, n 8: 13.9 us, 20.5 by 256, 200 by 1,024).
constexpr int kSelectRanked = 128;
constexpr int kFewLoads = 16;      // loads that one wave ranks; their elements cannot overflow the list
static_assert(kFewLoads * 8 <= kSelectRanked && kSelectRanked <= kSelectList, "what one wave ranks is never too long");
constexpr int kRankLanes = 8;      // lanes that count the larger ones of one element together
// Up to so many of 64 values the n-th largest is a good bound: some 45 elements reach it where n
// is 32.  All 64 are reached by hundreds, so more of them take 256 values (64 candidates of 64 x
// 16 rows of 65,536 bf16: 40.5 us by 256, 94 by 64, most of whose bounds are raised again; 33
// candidates 32.2 and 31.0).
constexpr int kFewCandidates = 32;
// The join ranks up to so many, and raises its bound above that (4 rows of 129,280 bf16, one token
// allowed and the others -1e4, 8 candidates: 31 us, 263 where up to 2,048 were ranked).
constexpr int kMergeRanked = 256;
constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.44269504088896341f;

// Unsigned numbers in the order of the floats (no NaN).
__device__ __forceinline__ uint32_t in_order(float x) {
  const uint32_t b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_order(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ uint32_t high_in_order(double x) {
  const uint32_t h = (uint32_t)__double2hiint(x);
  return (h & 0x80000000u) ? ~h : h | 0x80000000u;
}

// Larger logits first, then lower tokens.  (x + 0 makes -0 and 0 one value.)
__device__ __forceinline__ unsigned long long select_key(float x, int token) {
  return (unsigned long long)in_order(x + 0.0f) << 32 | (uint32_t)~token;
}
__device__ __forceinline__ float key_logit(unsigned long long key) { return from_order((uint32_t)(key >> 32)); }
__device__ __forceinline__ int key_token(unsigned long long key) { return (int)~(uint32_t)key; }

// The largest bound of `bits` (even) leading bits that at least n lanes' values reach (n <= 64; 0
// if fewer than n lanes have any): two bits a step, since every step waits for the last.
__device__ __forceinline__ uint32_t bound_of_lanes(uint32_t value, int n, int bits) {
  uint32_t bound = 0;
  for (int b = 30; b >= 32 - bits; b -= 2) {
    const uint32_t one = bound | 1u << b, two = bound | 2u << b, three = bound | 3u << b;
    const int n1 = __popcll(__ballot(value >= one)), n2 = __popcll(__ballot(value >= two)),
              n3 = __popcll(__ballot(value >= three));
    bound = n3 >= n ? three : n2 >= n ? two : n1 >= n ? one : bound;
  }
  return bound;
}

// The same for 256 values, four of them a lane.
__device__ __forceinline__ uint32_t bound_of_four(uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3, int n, int bits) {
  uint32_t bound = 0;
  for (int b = 31; b >= 32 - bits; --b) {
    const uint32_t next = bound | 1u << b;
    const int count = __popcll(__ballot(v0 >= next)) + __popcll(__ballot(v1 >= next)) + __popcll(__ballot(v2 >= next)) +
                      __popcll(__ballot(v3 >= next));
    if (count >= n) bound = next;
  }
  return bound;
}

// Reductions over a wave by data-parallel moves (the last lane has the result, lanes without a
// source take `none`), a third of the latency of six exchanges through LDS.
template <int CTRL, int ROWS>
__device__ __forceinline__ float moved(float none, float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(none), __float_as_int(v), CTRL, ROWS, 0xf, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double none, double v) {
  const int lo = __builtin_amdgcn_update_dpp(__double2loint(none), __double2loint(v), CTRL, ROWS, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(__double2hiint(none), __double2hiint(v), CTRL, ROWS, 0xf, false);
  return __hiloint2double(hi, lo);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ int moved(int none, int v) {
  return __builtin_amdgcn_update_dpp(none, v, CTRL, ROWS, 0xf, false);
}
template <typename V, typename F>
__device__ __forceinline__ V of_wave(V v, V none, F f) {
  v = f(v, moved<0x111, 0xf>(none, v));  // row_shr 1, 2, 4, 8
  v = f(v, moved<0x112, 0xf>(none, v));
  v = f(v, moved<0x114, 0xf>(none, v));
  v = f(v, moved<0x118, 0xf>(none, v));
  v = f(v, moved<0x142, 0xa>(none, v));  // row_bcast 15, 31
  return f(v, moved<0x143, 0xc>(none, v));
}
__device__ __forceinline__ float last_lane(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ int last_lane(int v) { return __builtin_amdgcn_readlane(v, 63); }
__device__ __forceinline__ double last_lane(double v) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), 63), __builtin_amdgcn_readlane(__double2loint(v), 63));
}
// (A NaN stays one.)
__device__ __forceinline__ float max_of_wave(float v) {
  return last_lane(of_wave(v, -INFINITY, [](float a, float b) { return __builtin_elementwise_maximum(a, b); }));
}
template <typename V>
__device__ __forceinline__ V sum_of_wave(V v) {
  return last_lane(of_wave(v, (V)0, [](V a, V b) { return a + b; }));
}
// Over groups of 8 lanes, in all of them: quad_perm 1, 0, 3, 2; quad_perm 2, 3, 0, 1; row_half_mirror.
template <typename V, typename F>
__device__ __forceinline__ V of_eight(V v, F f) {
  v = f(v, moved<0xB1, 0xf>(v, v));
  v = f(v, moved<0x4E, 0xf>(v, v));
  return f(v, moved<0x141, 0xf>(v, v));
}
__device__ __forceinline__ float max_of_eight(float v) {
  return of_eight(v, [](float a, float b) { return __builtin_elementwise_maximum(a, b); });
}
template <typename V>
__device__ __forceinline__ V sum_of_eight(V v) {
  return of_eight(v, [](V a, V b) { return a + b; });
}

// kVec logits from element e of a row on, or those below `end` and -inf for the others.  A lane's
// elements go by their place in the row, not by the row's place in its 16-byte lines (a load may
// start at any element), so that equal rows have equal sums, and beams with equal totals keep
// their order.
template <typename T>
struct Logits;
template <>
struct Logits<float> {
  static constexpr int kVec = 4, kWaves = 5;
  typedef float raw_t __attribute__((ext_vector_type(4)));
  typedef raw_t anywhere_t __attribute__((aligned(4)));
  raw_t raw;
  __device__ __forceinline__ void load(const float* x, int e) {
    raw = __builtin_nontemporal_load(reinterpret_cast<const anywhere_t*>(x + e));
  }
  __device__ __forceinline__ void load_below(const float* x, int e, int end) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) raw[i] = e + i < end ? x[e + i] : -INFINITY;
  }
  __device__ __forceinline__ float at(int i) const { return raw[i]; }
  // at(i) for an i that is not known before, in LDS
  __device__ __forceinline__ float pick(int i) const { return reinterpret_cast<const float*>(&raw)[i]; }
  __device__ __forceinline__ void again() {}
};
template <>
struct Logits<uint16_t> {  // bf16
  static constexpr int kVec = 8, kWaves = 8;
  typedef uint32_t raw_t __attribute__((ext_vector_type(4)));
  typedef raw_t anywhere_t __attribute__((aligned(2)));
  raw_t raw;
  __device__ __forceinline__ void load(const uint16_t* x, int e) {
    raw = __builtin_nontemporal_load(reinterpret_cast<const anywhere_t*>(x + e));
  }
  __device__ __forceinline__ void load_below(const uint16_t* x, int e, int end) {
#pragma unroll
    for (int i = 0; i < kVec; i += 2) {
      const uint32_t lo = e + i < end ? x[e + i] : 0xFF80u;
      const uint32_t hi = e + i + 1 < end ? x[e + i + 1] : 0xFF80u;
      raw[i / 2] = hi << 16 | lo;
    }
  }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i & 1 ? raw[i / 2] & 0xFFFF0000u : raw[i / 2] << 16);
  }
  __device__ __forceinline__ float pick(int i) const {
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(&raw)[i] << 16);
  }
  // Widened logits are not kept from one pass to the next: 64 registers instead of 32 would cost
  // half of the waves.
  __device__ __forceinline__ void again() { asm volatile("" : "+v"(raw)); }
};

// A piece whose maximum m is below kFar takes the float next to m log2e off its exponents (in powers
// of two), and is off by its rounding, at most 2^-14, whose square is left out of the correction.
constexpr float kFar = 1024.0f;
__device__ __forceinline__ float select_center(float m) { return m * kLog2e; }

// Beams whose logits are not read: done, or without a finite score.
__device__ __forceinline__ bool beam_is_live(const SelectArgs& a, int row) {
  return (a.done == nullptr || a.done[row] == 0) && isfinite(a.scores[row]);
}

// Logits are read past the caches (2,048 rows of 129,280 fp32: 175 -> 157 us).  bf16 runs 8 waves
// a SIMD: 64 registers, and 8 workgroups' lists in a CU's LDS; fp32 has twice the loads to list,
// which leave 5 workgroups, and these read faster than 8 (154 against 157 us; bf16 by 5, 512 rows
// of 65,537: 26 against 24).
template <typename T, int NV>
__global__ __launch_bounds__(kSelectThreads, Logits<T>::kWaves) void beam_select_rows_kernel(SelectArgs a) {
  constexpr int kVec = Logits<T>::kVec, kSelectLoads = kSelectHeld / kVec;
  const int row = (int)(blockIdx.x / (unsigned)a.splits), piece = (int)(blockIdx.x % (unsigned)a.splits);
  if (!beam_is_live(a, row)) return;
  __shared__ float lane_max[4][64];
  __shared__ float wave_sum[4];
  __shared__ Logits<T> load_list[kSelectLoads];
  __shared__ int load_at[kSelectLoads];
  __shared__ unsigned long long list[kSelectList];
  __shared__ int loads, listed;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const T* x = static_cast<const T*>(a.logits) + row * a.ld;
  constexpr int kBlock = kSelectThreads * kVec;
  const int first = piece * NV * kBlock, end = min(a.V, first + NV * kBlock), e0 = first + tid * kVec;
  Logits<T> v[NV];
  if (end - first == NV * kBlock) {
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j].load(x, e0 + j * kBlock);
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (e0 + j * kBlock + kVec <= end)
        v[j].load(x, e0 + j * kBlock);
      else
        v[j].load_below(x, e0 + j * kBlock, end);
    }
  }
  if (tid == 0) loads = listed = 0;

  // a NaN makes its maxima NaN, +inf infinite: rows without candidates
  float most[NV];
  float mine = -INFINITY;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    most[j] = v[j].at(0);
#pragma unroll
    for (int i = 1; i < kVec; ++i) most[j] = __builtin_elementwise_maximum(most[j], v[j].at(i));
    mine = __builtin_elementwise_maximum(mine, most[j]);
    v[j].again();
  }
  lane_max[wave][lane] = mine;
  __syncthreads();
  const float m0 = lane_max[0][lane], m1 = lane_max[1][lane], m2 = lane_max[2][lane], m3 = lane_max[3][lane];
  const float of_lane = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m0, m1), __builtin_elementwise_maximum(m2, m3));
  const float m = max_of_wave(of_lane);
  // the bound keeps 16 bits: exact for bf16, and 2^-8 below the n-th of the maxima for fp32
  const uint32_t reach = a.n <= kFewCandidates
                             ? bound_of_lanes(in_order(of_lane), a.n, 16)
                             : bound_of_four(in_order(m0), in_order(m1), in_order(m2), in_order(m3), a.n, 16);
  const float bound = reach <= in_order(kLowest) ? kLowest : from_order(reach);

  // exp(x - m) as 2^(x log2e - c), c the float next to m log2e: one fma, rounded by 2^-24 of the
  // exponent; the merge makes up for c's own rounding.  Far from zero, as 2^((x - m) log2e).
  const float c = select_center(m);
  const bool far = fabsf(m) >= kFar;
  const float base = m == -INFINITY ? 0.0f : m;
  float sum[2] = {0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (most[j] >= bound) {
      const int place = atomicAdd(&loads, 1);
      if (place < kSelectLoads) {
        load_list[place] = v[j];
        load_at[place] = e0 + j * kBlock;
      }
    }
    if (!far) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) sum[i & 1] += __builtin_amdgcn_exp2f(__builtin_fmaf(v[j].at(i), kLog2e, -c));
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) sum[i & 1] += __builtin_amdgcn_exp2f((v[j].at(i) - base) * kLog2e);
    }
  }
  const float s = sum_of_wave(sum[0] + sum[1]);
  if (lane == 0) wave_sum[wave] = s;
  __syncthreads();
  if (tid == 0) a.parts[blockIdx.x] = make_float2(m, (wave_sum[0] + wave_sum[1]) + (wave_sum[2] + wave_sum[3]));
  unsigned long long* out = a.keys + (int64_t)blockIdx.x * a.n;
  if (loads <= kSelectLoads) {
    // one wave is enough for few of them, and needs no barriers
    const int workers = loads <= kFewLoads ? 64 : kSelectThreads;
    if (tid >= workers) return;
    for (int i = tid; i < loads * kVec; i += workers) {
      const float f = load_list[i / kVec].pick(i % kVec);
      if (f >= bound) {
        const int place = atomicAdd(&listed, 1);
        if (place < kSelectList) list[place] = select_key(f, load_at[i / kVec] + i % kVec);
      }
    }
    if (workers == 64)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    else
      __syncthreads();
    const int reached = listed;
    if (reached <= kSelectRanked) {
      for (int i = tid / kRankLanes; i < reached; i += workers / kRankLanes) {
        const unsigned long long key = list[i];
        int rank = 0;
        for (int k = tid % kRankLanes; k < reached; k += kRankLanes) rank += list[k] > key ? 1 : 0;
        rank = sum_of_eight(rank);
        if (rank < a.n && tid % kRankLanes == 0) out[rank] = key;
      }
      for (int i = reached + tid; i < a.n; i += workers) out[i] = 0;
      return;
    }
  }
  // The bound for all 32 bits, again from the lanes' maxima: n elements at least reach lo, fewer
  // reach hi.  Few may reach it by now; where it is a mask's value, it is the n-th largest itself.
  if (!(m < INFINITY)) {  // a row without candidates
    for (int i = tid; i < a.n; i += kSelectThreads) out[i] = 0;
    return;
  }
  __shared__ int reached_by[2][4];
  const uint32_t u0 = in_order(lane_max[0][lane]), u1 = in_order(lane_max[1][lane]), u2 = in_order(lane_max[2][lane]),
                 u3 = in_order(lane_max[3][lane]);
  uint32_t lo = a.n <= kFewCandidates ? bound_of_lanes(max(max(u0, u1), max(u2, u3)), a.n, 32)
                                      : bound_of_four(u0, u1, u2, u3, a.n, 32);
  lo = max(lo, in_order(kLowest));
  uint32_t hi = in_order(m) + 1u, mid = lo;
  bool few = false;
  for (int step = 0; hi - lo > 1u && !few; ++step) {
    const float t = from_order(mid);
    int count = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      v[j].again();
#pragma unroll
      for (int i = 0; i < kVec; ++i) count += v[j].at(i) >= t ? 1 : 0;
    }
    count = sum_of_wave(count);
    if (lane == 0) reached_by[step & 1][wave] = count;
    __syncthreads();  // (the next step writes the other half, so one is enough)
    const int* of = reached_by[step & 1];
    count = (of[0] + of[1]) + (of[2] + of[3]);
    if (count >= a.n) {
      lo = mid;
      few = count <= kSelectRanked;
    } else {
      hi = mid;
    }
    mid = step == 0 ? lo + 1u : lo + (hi - lo) / 2u;
  }
  // elements that reach lo, if they are few, else those above it: fewer than n (a comparison of
  // floats, to which zeros of both signs are equal)
  const float equal = from_order(lo);
  __shared__ int equals[NV][4];
  __syncthreads();  // the lists' first form is read
  if (tid == 0) listed = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    v[j].again();
    int count = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const float f = v[j].at(i);
      if (few ? f >= equal : f > equal) {
        const int place = atomicAdd(&listed, 1);
        list[place] = select_key(f, e0 + j * kBlock + i);
      }
      count += f == equal ? 1 : 0;
    }
    count = sum_of_wave(count);
    if (lane == 0) equals[j][wave] = count;
  }
  __syncthreads();
  const int above = listed;
  for (int i = tid / kRankLanes; i < above; i += kSelectThreads / kRankLanes) {
    const unsigned long long key = list[i];
    int rank = 0;
    for (int k = tid % kRankLanes; k < above; k += kRankLanes) rank += list[k] > key ? 1 : 0;
    rank = sum_of_eight(rank);
    if (rank < a.n && tid % kRankLanes == 0) out[rank] = key;
  }
  if (few) return;
  // equal ones by token: by block, then lane, then place in the lane's load
  int rank0 = above;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    int rank = rank0;
    for (int w = 0; w < 4; ++w) {
      if (w < wave) rank += equals[j][w];
      rank0 += equals[j][w];
    }
    if (rank >= a.n) continue;
    v[j].again();
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const unsigned long long same = __ballot(v[j].at(i) == equal);
      rank += __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (v[j].at(i) == equal) {
        if (rank < a.n) out[rank] = select_key(equal, e0 + j * kBlock + i);
        ++rank;
      }
  }
}

// What a request's beams add to their logits: total = (score + (x - most)) - norm.
struct MergeBeams {
  double score[64], most[64], norm[64];
  int kind[64];  // 0: no candidates, 1: live, 2: done
};

__device__ __forceinline__ double beam_total(const MergeBeams& s, int b, unsigned long long key) {
  return (s.score[b] + ((double)key_logit(key) - s.most[b])) - s.norm[b];
}

// The order of candidates in two whole numbers: totals (-0 as 0), and among equal ones lower beams,
// larger logits, lower tokens (of 24 bits).
__device__ __forceinline__ unsigned long long total_in_order(double t) {
  const unsigned long long b = (unsigned long long)__double_as_longlong(t + 0.0);
  return (b >> 63) != 0 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ unsigned long long place_in_order(int b, unsigned long long key) {
  return (unsigned long long)(63 - b) << 56 | (key >> 32) << 24 | (key & 0xFFFFFFu);
}

__device__ __forceinline__ bool goes_before(double ta, int ba, unsigned long long ka, double tb, int bb,
                                            unsigned long long kb) {
  return ta > tb || (ta == tb && (ba < bb || (ba == bb && ka > kb)));
}

// Keys a thread keeps in registers.
constexpr int kMergeKeys = 8;

template <int THREADS>
__global__ __launch_bounds__(THREADS) void beam_select_merge_kernel(SelectArgs a) {
  __shared__ MergeBeams beams;
  __shared__ uint32_t slot_max[256];
  __shared__ double totals[kMergeRanked];
  __shared__ unsigned long long keys[kMergeRanked];
  __shared__ uint8_t of_beam[kMergeRanked];
  __shared__ int listed;
  const int g = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int S = a.splits, K = a.K, n = a.n;
  // place i of the request's keys is the (i / pieces)-th of piece i % pieces: the largest first
  const int pieces = K * S, places = pieces * n;
  const unsigned long long* all = a.keys + (int64_t)g * places;
  unsigned long long mine[kMergeKeys];  // (of beams that are not live: not written, and not looked at)
  int piece_of[kMergeKeys], slot_of[kMergeKeys];
  {
    int piece = tid % pieces, order = tid / pieces;
    const int step = THREADS % pieces, steps = THREADS / pieces;
#pragma unroll
    for (int q = 0; q < kMergeKeys; ++q) {
      piece_of[q] = piece;
      slot_of[q] = (piece + 13 * order) & 255;
      mine[q] = order < n ? all[piece * n + order] : 0;
      piece += step;
      order += steps;
      if (piece >= pieces) {
        piece -= pieces;
        ++order;
      }
    }
  }
  if (tid == 0) listed = 0;
  if (tid < 256) slot_max[tid] = 0;
  // a beam a wave, or eight where a row is at most eight pieces (64 beams of one piece: a call of
  // 14.6 us by one, 8.2 by eight)
  const bool eight = S <= 8;
  const int width = eight ? 8 : 64, at = lane % width;
  for (int b0 = wave * (64 / width); b0 < K; b0 += THREADS / width) {
    const int b = b0 + lane / width;
    const int row = g * K + min(b, K - 1);
    const float2* part = a.parts + (int64_t)row * S;
    float2 p = at < S ? part[at] : make_float2(-INFINITY, 0.0f);  // (of a beam that is not live: any bits)
    const float score = a.scores[row];
    const bool done = a.done != nullptr && a.done[row] != 0;
    float m = p.x;
    for (int i = at + 64; i < S; i += 64) m = __builtin_elementwise_maximum(m, part[i].x);
    m = eight ? max_of_eight(m) : max_of_wave(m);
    double z = 0.0;
    for (int i = at; i < S; i += 64) {
      if (i >= 64) p = part[i];
      // a piece's sum is of 2^(x log2e - c), with the constant as fp32 has it.  Its scale 2^(d log2e),
      // d <= 0, is an exponential of fp32: a unit of its own, and 2^-24 |d| each of the difference's
      // and the product's rounding.  They count e^d times: some 2^-23 of the whole sum at most,
      // no more than the piece's own exponentials are off
      const double shift = fabsf(p.x) < kFar ? (double)select_center(p.x) - (double)p.x * (double)kLog2e : 0.0;
      const float scale = __builtin_amdgcn_exp2f((p.x - m) * kLog2e);
      z += (double)p.y * (double)scale * (1.0 + shift * 0.6931471805599453);
    }
    z = eight ? sum_of_eight(z) : sum_of_wave(z);
    if (at == 0 && b < K) {
      beams.score[b] = (double)score;
      beams.most[b] = (double)m;
      beams.norm[b] = log(z);
      beams.kind[b] = !isfinite(score) ? 0 : done ? 2 : isfinite(m) && isfinite(z) ? 1 : 0;
    }
  }
  __syncthreads();

  // A bound that n of 64 (or 256) slots reach, by the 12 leading bits of the totals' mantissas.
  // Every key counts for a slot by its piece and its rank there, so that the slots have equal
  // shares of the best keys even where one beam has them all.
  double total[kMergeKeys];
#pragma unroll
  for (int q = 0; q < kMergeKeys; ++q) {
    if (mine[q] == 0) continue;
    piece_of[q] /= S;  // the beam
    if (beams.kind[piece_of[q]] != 1) {
      mine[q] = 0;
      continue;
    }
    total[q] = beam_total(beams, piece_of[q], mine[q]);
    atomicMax(&slot_max[slot_of[q]], high_in_order(total[q]));
  }
  __syncthreads();
  const uint32_t s0 = slot_max[lane], s1 = slot_max[64 + lane], s2 = slot_max[128 + lane], s3 = slot_max[192 + lane];
  const uint32_t bound = n <= kFewCandidates ? bound_of_lanes(max(max(s0, s1), max(s2, s3)), n, 24)
                                             : bound_of_four(s0, s1, s2, s3, n, 24);

  auto push = [&](double total, int b, unsigned long long key) {
    const int place = atomicAdd(&listed, 1);
    if (place < kMergeRanked) {
      totals[place] = total;
      keys[place] = key;
      of_beam[place] = (uint8_t)b;
    }
  };
#pragma unroll
  for (int q = 0; q < kMergeKeys; ++q)
    if (mine[q] != 0 && high_in_order(total[q]) >= bound) push(total[q], piece_of[q], mine[q]);
  // the keys that no thread has: a piece's descend, so it is left at the first below the bound
  if (places > kMergeKeys * THREADS) {
    for (int piece = tid; piece < pieces; piece += THREADS) {
      const int b = piece / S;
      if (beams.kind[b] != 1) continue;
      const int known = piece < kMergeKeys * THREADS ? (kMergeKeys * THREADS - piece + pieces - 1) / pieces : 0;
      for (int order = known; order < n; ++order) {
        const unsigned long long key = all[(int64_t)piece * n + order];
        if (key == 0) break;
        const double t = beam_total(beams, b, key);
        if (high_in_order(t) < bound) break;
        push(t, b, key);
      }
    }
  }
  if (tid < K && beams.kind[tid] == 2) push(beams.score[tid], tid, select_key(0.0f, a.end_token));
  __syncthreads();

  auto write = [&](int r, double total, int b, unsigned long long key) {
    const int64_t at = (int64_t)g * n + r;
    const int token = key_token(key);
    a.tokens[at] = token;
    a.parents[at] = b;
    a.out_scores[at] = (float)total;
    if (a.out_done != nullptr) a.out_done[at] = beams.kind[b] == 2 || token == a.end_token ? 1 : 0;
  };
  auto write_none = [&](int r) {
    const int64_t at = (int64_t)g * n + r;
    a.tokens[at] = -1;
    a.parents[at] = -1;
    a.out_scores[at] = -INFINITY;
    if (a.out_done != nullptr) a.out_done[at] = 0;
  };
  int count = listed;
  if (count > kMergeRanked) {
    // Totals that agree in the bound's bits, as those of masked tokens do.  The bound is raised by
    // bisection, counting again, until few reach it or it is the n-th largest total, and then among
    // the candidates of that total by their places, which are all different.
    __shared__ int counts[2][THREADS / 64];
    __shared__ unsigned long long ends[2][THREADS / 64];
    int turn = 0;
    auto count_all = [&](int c) {
      c = sum_of_wave(c);
      if (lane == 0) counts[turn][wave] = c;
      __syncthreads();  // (the next count writes the other half, so one is enough)
      int sum = 0;
      for (int w = 0; w < THREADS / 64; ++w) sum += counts[turn][w];
      turn ^= 1;
      return sum;
    };
    // candidates whose totals reach `least`
    auto each = [&](unsigned long long least, auto f) {
#pragma unroll
      for (int q = 0; q < kMergeKeys; ++q)
        if (mine[q] != 0 && total_in_order(total[q]) >= least) f(total[q], piece_of[q], mine[q]);
      if (places > kMergeKeys * THREADS) {
        for (int piece = tid; piece < pieces; piece += THREADS) {
          const int b = piece / S;
          if (beams.kind[b] != 1) continue;
          const int known = piece < kMergeKeys * THREADS ? (kMergeKeys * THREADS - piece + pieces - 1) / pieces : 0;
          for (int order = known; order < n; ++order) {
            const unsigned long long key = all[(int64_t)piece * n + order];
            if (key == 0) break;
            const double t = beam_total(beams, b, key);
            if (total_in_order(t) < least) break;
            f(t, b, key);
          }
        }
      }
      if (tid < K && beams.kind[tid] == 2 && total_in_order(beams.score[tid]) >= least)
        f(beams.score[tid], tid, select_key(0.0f, a.end_token));
    };
    // the least lo and the largest hi of the workgroup
    auto ends_of = [&](unsigned long long& lo, unsigned long long& hi) {
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) {
        const unsigned long long l = __shfl_xor(lo, off, 64), h = __shfl_xor(hi, off, 64);
        lo = l < lo ? l : lo;
        hi = h > hi ? h : hi;
      }
      __syncthreads();  // earlier ends are read
      if (lane == 0) ends[0][wave] = lo, ends[1][wave] = hi;
      __syncthreads();
      for (int w = 0; w < THREADS / 64; ++w) {
        lo = ends[0][w] < lo ? ends[0][w] : lo;
        hi = ends[1][w] > hi ? ends[1][w] : hi;
      }
    };
    // lo, which at least `want` of the visited numbers reach, is raised below hi, which `above` do,
    // fewer: until at most `room` reach it (true), or it is the want-th largest itself.  Numbers lie
    // in clusters (the totals of a beam's masked tokens, the places of a beam), so both ends go
    // to the next numbers now and then.
    auto raise = [&](unsigned long long& lo, int first, int want, int room, int& above, auto visit) {
      unsigned long long hi = ~0ull, mid = 0;
      above = 0;
      for (int step = 0;; ++step) {
        if (step % 8 == 0) {
          unsigned long long l = ~0ull, h = 0;
          visit(lo, [&](unsigned long long v) {
            if (v < lo || v >= hi) return;
            l = v < l ? v : l;
            h = v > h ? v : h;
          });
          ends_of(l, h);
          lo = l;
          hi = h + 1;
          mid = step == 0 ? lo + first : lo + (hi - lo) / 2;
        }
        if (hi <= lo || hi - lo == 1) return false;
        int c = 0;
        visit(mid, [&](unsigned long long v) { c += v >= mid ? 1 : 0; });
        c = count_all(c);
        if (c >= want) {
          lo = mid;
          if (c <= room) return true;
        } else {
          hi = mid;
          above = c;
        }
        mid = lo + (hi - lo) / 2;
      }
    };
    unsigned long long cut = (unsigned long long)bound << 32, place = 0;
    int above, ahead;
    // (the first step asks whether the least total is the n-th itself)
    if (!raise(cut, 1, n, kMergeRanked, above, [&](unsigned long long least, auto f) {
          each(least, [&](double t, int, unsigned long long) { f(total_in_order(t)); });
        }))
      raise(place, 0, n - above, kMergeRanked - above, ahead, [&](unsigned long long, auto f) {
        each(cut, [&](double t, int b, unsigned long long key) {
          if (total_in_order(t) == cut) f(place_in_order(b, key));
        });
      });
    if (tid == 0) listed = 0;
    __syncthreads();
    each(cut, [&](double t, int b, unsigned long long key) {
      if (total_in_order(t) != cut || place_in_order(b, key) >= place) push(t, b, key);
    });
    __syncthreads();
    count = listed;
  }
  for (int i = tid / kRankLanes; i < count; i += THREADS / kRankLanes) {
    const double total = totals[i];
    const unsigned long long key = keys[i];
    const int b = of_beam[i];
    int rank = 0;
    for (int k = tid % kRankLanes; k < count; k += kRankLanes)
      rank += goes_before(totals[k], of_beam[k], keys[k], total, b, key) ? 1 : 0;
    rank = sum_of_eight(rank);
    if (rank < n && tid % kRankLanes == 0) write(rank, total, b, key);
  }
  for (int r = count + tid; r < n; r += THREADS) write_none(r);
}

// ---------------------------------------------------------------------------
// Pieces of a row of V elements, of up to nv blocks each.
static int select_splits(int V, int vec, int nv) {
  const int per = nv * vec * kSelectThreads;
  return (V + per - 1) / per;
}

// Loads a lane: as many as leave this many workgroups, up to 8 and to what a row takes.
constexpr int kSelectGroups = 1024;

static int select_loads(int64_t rows, int V, int vec) {
  int nv = 8;
  while (nv > 1 && (rows * select_splits(V, vec, nv) < kSelectGroups || select_splits(V, vec, nv / 2) == 1)) nv >>= 1;
  return nv;
}

// Pieces that calls of up to G requests can have, in either type.
static int64_t select_pieces(int64_t rows, int V) {
  int64_t most = 0;
  for (int vec = 4; vec <= 8; vec += 4)
    for (int nv = 1; nv <= 8; nv <<= 1) {
      // rows for which nv is taken: fewer than twice the loads would need
      int64_t r = rows;
      if (nv < 8) r = std::min(r, (int64_t)(kSelectGroups - 1) / select_splits(V, vec, 2 * nv));
      most = std::max(most, r * select_splits(V, vec, nv));
    }
  return most;
}

int64_t beam_select_workspace_bytes(int32_t G, int32_t K, int32_t V, int32_t n) {
  return select_pieces((int64_t)G * K, V) * (int64_t)(sizeof(float2) + n * sizeof(unsigned long long));
}

template <typename T>
static void launch_select_rows(const SelectArgs& a, int nv, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)a.G * a.K * a.splits)), block(kSelectThreads);
  switch (nv) {
    case 1: hipLaunchKernelGGL((beam_select_rows_kernel<T, 1>), grid, block, 0, stream, a); break;
    case 2: hipLaunchKernelGGL((beam_select_rows_kernel<T, 2>), grid, block, 0, stream, a); break;
    case 4: hipLaunchKernelGGL((beam_select_rows_kernel<T, 4>), grid, block, 0, stream, a); break;
    default: hipLaunchKernelGGL((beam_select_rows_kernel<T, 8>), grid, block, 0, stream, a); break;
  }
}

hipError_t launch_beam_select(const SelectArgs& args, hipStream_t stream) {
  (void)hipGetLastError();  // drop a stale error another library left on this thread
  SelectArgs a = args;
  if (a.G == 0) return hipSuccess;
  const int vec = a.f32 ? 4 : 8;
  const int nv = select_loads((int64_t)a.G * a.K, a.V, vec);
  a.splits = select_splits(a.V, vec, nv);
  const int64_t pieces = (int64_t)a.G * a.K * a.splits;
  a.keys = static_cast<unsigned long long*>(a.work);
  a.parts = reinterpret_cast<float2*>(a.keys + pieces * a.n);
  if (a.f32)
    launch_select_rows<float>(a, nv, stream);
  else
    launch_select_rows<uint16_t>(a, nv, stream);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if ((int64_t)a.K * a.splits * a.n > kMergeKeys * 512)
    hipLaunchKernelGGL(beam_select_merge_kernel<1024>, dim3(a.G), dim3(1024), 0, stream, a);
  else
    hipLaunchKernelGGL(beam_select_merge_kernel<512>, dim3(a.G), dim3(512), 0, stream, a);
  return hipGetLastError();
}

}  // namespace engram
