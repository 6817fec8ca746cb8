// Attention over the paged int8 cache: per query row i of sequence b and head h,
// over the cached rows j < length[b] (causal: j <= length[b] - rows + i)
//   s_j = (q . code_j) s_k / sqrt(d) - penalty(|t_q - t_j|),
//   O = sum_j exp(s_j) code_j s_v / sum_j exp(s_j),   LSE = log sum_j exp(s_j);
// a row that sees no key gets O = 0 and LSE = -inf.
//
// The plainest form: one warp per query row and head, 32 keys at a time (one
// per lane for the scores, d / 32 columns per lane for the values).
#include <cuda_bf16.h>

#include "cache.cuh"

namespace h3 {
namespace {

template <int D>
__global__ void __launch_bounds__(128) rows_kernel(const CacheAttnParams p) {
  __shared__ float qs[4][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * 4 + warp, h = blockIdx.y, hk = h / p.group;
  int b = -1, i = 0, n = 0;
  for (int x = 0; x < p.b.B && b < 0; ++x) {
    const SeqRows s = seq_rows(p.b, x, p.status);
    if (t >= s.first && t < s.first + s.n) {
      b = x;
      i = t - s.first;
      n = s.n;
    }
  }
  if (b < 0 || t >= p.b.T) return;
  const int len = seq_length(p.b, b, p.status);
  const int seen = p.causal ? max(0, len - n + i + 1) : len;
  for (int c = lane; c < D; c += 32)
    qs[warp][c] = __uint_as_float((uint32_t)p.q[h * p.q_head + t * p.q_row + c] << 16);
  __syncwarp();
  const float tq = p.q_times != nullptr ? p.q_times[t] : NAN;
  float m = -INFINITY, l = 0.0f, o[D / 32] = {};
  for (int j0 = 0; j0 < seen; j0 += 32) {
    const int page = page_id(p.c, p.b, b, j0 / kBlock, p.status);
    if (page < 0) continue;
    const size_t at = (size_t)page * p.c.H + hk;
    const int8_t* k = p.c.k + at * kBlock * D + (size_t)(j0 % kBlock + lane) * D;
    float s = -INFINITY;
    if (j0 + lane < seen) {
      float dot = 0.0f;
      for (int c = 0; c < D; ++c) dot = fmaf((float)k[c], qs[warp][c], dot);
      s = dot * (p.c.k_scale[at] * p.scale_log2);
      if (p.q_times != nullptr) {
        const float dt = fabsf(tq - p.c.times[(size_t)page * kBlock + j0 % kBlock + lane]);
        const float e = fmaxf(dt - p.window, 0.0f) * p.inv_falloff;
        s -= fminf(p.strength_log2 * e * e, p.cap_log2);
      }
    }
    float top = s;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
    const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.0f : mn;
    const float alpha = exp2f(m - base), e = exp2f(s - base);
    m = mn;
    l = l * alpha + e;
    const float pv = e * p.c.v_scale[at];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[c] *= alpha;
    const int8_t* v = p.c.v + at * kBlock * D + (size_t)(j0 % kBlock) * D;
    const int live = min(32, seen - j0);
    for (int x = 0; x < live; ++x) {
      const float w = __shfl_sync(0xFFFFFFFFu, pv, x);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) o[c] = fmaf(w, (float)v[x * D + c * 32 + lane], o[c]);
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t* out = p.o + ((size_t)h * p.b.T + t) * D;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    const __nv_bfloat16 y = __float2bfloat16_rn(o[c] * inv);
    out[c * 32 + lane] = *reinterpret_cast<const uint16_t*>(&y);
  }
  if (p.lse != nullptr && lane == 0) p.lse[(size_t)h * p.b.T + t] = (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_cache_attn(const CacheAttnParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.b.T + 3) / 4), (unsigned)p.H);
  if (p.c.d == 64) rows_kernel<64><<<grid, 128, 0, stream>>>(p);
  else rows_kernel<128><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace h3
