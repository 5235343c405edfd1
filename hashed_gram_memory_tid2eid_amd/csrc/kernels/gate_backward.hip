// gate_backward.hip -- the gradient of the sigmoid-gated residual add of gate.hip.
// Included into engram_device.hip after gate.hip, whose helpers it uses.
//
//   z_s = <x_s, v> r,  g_s = sigmoid(z_s),  y_s = x_s + k g_s v,   r = 1 / sqrt(hidden), k = keep
//   e_s = k <dy_s, v> g_s (1 - g_s) r
//   dx_s = dy_s + e_s v,   dv = sum_s (k g_s dy_s + e_s x_s)
//
// One workgroup per token holds the token's v (fp32) and its four streams of x and dy
// (bf16) in registers, so every byte is read once and written once; the eight dot
// products are reduced by wave shuffles and a fixed-order sum over the waves in LDS
// (deterministic).  The gate is recomputed from x and v: keeping it would save no read,
// since dx and dv need x and v anyway.  A token with keep = 0 passes dy through and has
// dv = 0.  dx may be dy itself: a thread writes only where it alone has read.
//
// Memory bounds it: 16,384 tokens of 4 x 4,096 read 1.34 GB and write 0.81 GB in 323 us, 6.6 TB/s,
// with dx written past the caches (370 us with ordinary stores).

namespace engram {

template <int CPT, int THREADS>
__global__ __launch_bounds__(THREADS) void gate_backward_kernel(GateBackwardArgs a) {
  const int t = blockIdx.x;
  const bool kept = a.keep == nullptr || a.keep[t] != 0;
  const int tid = threadIdx.x;
  const int nchunks = a.hidden >> 3;
  const int64_t xbase = (int64_t)t * kHc * a.hidden;
  const unsigned short* xrow = static_cast<const unsigned short*>(a.x) + xbase;
  const unsigned short* dyrow = static_cast<const unsigned short*>(a.dy) + xbase;
  unsigned short* dxrow = static_cast<unsigned short*>(a.dx) + xbase;
  const float* vrow = a.v + (int64_t)t * a.hidden;
  float* dvrow = a.dv + (int64_t)t * a.hidden;

  if (!kept) {  // uniform per workgroup
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int ch = tid + c * THREADS;
      if (ch >= nchunks) continue;
#pragma unroll
      for (int s = 0; s < kHc; ++s)
        *reinterpret_cast<g_u32x4*>(dxrow + (int64_t)s * a.hidden + ch * 8) =
            *reinterpret_cast<const g_u32x4*>(dyrow + (int64_t)s * a.hidden + ch * 8);
      *reinterpret_cast<g_f32x4*>(dvrow + ch * 8) = g_f32x4{};
      *reinterpret_cast<g_f32x4*>(dvrow + ch * 8 + 4) = g_f32x4{};
    }
    return;
  }

  g_f32x4 v[CPT][2];
  g_u32x4 x[kHc][CPT], dy[kHc][CPT];
  float dot[2 * kHc] = {};
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    const int ch = tid + c * THREADS;
    if (ch < nchunks) {
      v[c][0] = __builtin_nontemporal_load(reinterpret_cast<const g_f32x4*>(vrow + ch * 8));
      v[c][1] = __builtin_nontemporal_load(reinterpret_cast<const g_f32x4*>(vrow + ch * 8 + 4));
#pragma unroll
      for (int s = 0; s < kHc; ++s) {
        x[s][c] = __builtin_nontemporal_load(reinterpret_cast<const g_u32x4*>(xrow + (int64_t)s * a.hidden + ch * 8));
        dy[s][c] = __builtin_nontemporal_load(reinterpret_cast<const g_u32x4*>(dyrow + (int64_t)s * a.hidden + ch * 8));
      }
    } else {
      v[c][0] = v[c][1] = g_f32x4{};
#pragma unroll
      for (int s = 0; s < kHc; ++s) x[s][c] = dy[s][c] = g_u32x4{};
    }
  }
#pragma unroll
  for (int c = 0; c < CPT; ++c)
#pragma unroll
    for (int s = 0; s < kHc; ++s)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float v0 = v[c][w >> 1][2 * (w & 1)], v1 = v[c][w >> 1][2 * (w & 1) + 1];
        dot[s] = fmaf(bf16_lo(x[s][c][w]), v0, dot[s]);
        dot[s] = fmaf(bf16_hi(x[s][c][w]), v1, dot[s]);
        dot[kHc + s] = fmaf(bf16_lo(dy[s][c][w]), v0, dot[kHc + s]);
        dot[kHc + s] = fmaf(bf16_hi(dy[s][c][w]), v1, dot[kHc + s]);
      }

  __shared__ float part[THREADS / 64][2 * kHc];
#pragma unroll
  for (int i = 0; i < 2 * kHc; ++i) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) dot[i] += __shfl_xor(dot[i], off, 64);
  }
  if ((tid & 63) == 0) {
#pragma unroll
    for (int i = 0; i < 2 * kHc; ++i) part[tid >> 6][i] = dot[i];
  }
  __syncthreads();
  float g[kHc], e[kHc];
#pragma unroll
  for (int s = 0; s < kHc; ++s) {
    float z = part[0][s], d = part[0][kHc + s];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) {
      z += part[w][s];
      d += part[w][kHc + s];
    }
    // sigmoid(z) and sigmoid(-z) each from its own exponential: 1 - g would cancel at large z
    z *= a.inv_sqrt_hidden;
    g[s] = 1.0f / (1.0f + expf(-z));
    e[s] = d * g[s] * (1.0f / (1.0f + expf(z))) * a.inv_sqrt_hidden;
  }

#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    const int ch = tid + c * THREADS;
    if (ch >= nchunks) continue;
    g_f32x4 dv[2] = {};
#pragma unroll
    for (int s = 0; s < kHc; ++s) {
      g_u32x4 o;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int h = w >> 1, i0 = 2 * (w & 1), i1 = i0 + 1;
        const float dlo = bf16_lo(dy[s][c][w]), dhi = bf16_hi(dy[s][c][w]);
        o[w] = pack_bf16(fmaf(e[s], v[c][h][i0], dlo), fmaf(e[s], v[c][h][i1], dhi));
        dv[h][i0] = fmaf(g[s], dlo, fmaf(e[s], bf16_lo(x[s][c][w]), dv[h][i0]));
        dv[h][i1] = fmaf(g[s], dhi, fmaf(e[s], bf16_hi(x[s][c][w]), dv[h][i1]));
      }
      __builtin_nontemporal_store(o, reinterpret_cast<g_u32x4*>(dxrow + (int64_t)s * a.hidden + ch * 8));
    }
    *reinterpret_cast<g_f32x4*>(dvrow + ch * 8) = dv[0];
    *reinterpret_cast<g_f32x4*>(dvrow + ch * 8 + 4) = dv[1];
  }
}

hipError_t launch_gate_backward(const GateBackwardArgs& a, hipStream_t stream) {
  (void)hipGetLastError();  // drop a stale error another library left on this thread
  if (a.T == 0) return hipSuccess;
  const int nchunks = a.hidden / 8;
  const dim3 grid((unsigned)a.T);
  // one chunk of 8 elements per thread where the row allows it, as the forward gate
  if (nchunks <= 64)
    hipLaunchKernelGGL((gate_backward_kernel<1, 64>), grid, dim3(64), 0, stream, a);
  else if (nchunks <= 256)
    hipLaunchKernelGGL((gate_backward_kernel<1, 256>), grid, dim3(256), 0, stream, a);
  else if (nchunks <= 512)
    hipLaunchKernelGGL((gate_backward_kernel<1, 512>), grid, dim3(512), 0, stream, a);
  else if (nchunks <= 1024)
    hipLaunchKernelGGL((gate_backward_kernel<2, 512>), grid, dim3(512), 0, stream, a);
  else
    return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace engram
