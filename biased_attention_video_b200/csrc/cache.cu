// Paged int8 cache: appending keys and values (with the rotation of the keys
// on the way) and reading rows back.
//
// A page holds 64 consecutive rows of one sequence, all K/V heads, as int8
// codes [head][64][d] with one float32 scale per (page, head) for K and one
// for V: value = code * scale.  Appending rows to a page, in fp32 with every
// product, sum and quotient rounded to nearest (no fused multiply-add, so that
// the codes do not depend on how a compiler contracts):
//   K only:  y_i = x_i cos - x_j sin,  y_j = x_j cos + x_i sin  for pairs (i, j)
//   a  = max |y| over the new rows of the page and head
//   s' = max(s if the page holds earlier rows, a / 127, 2^-100)
//   code = clamp(rint(y * (1 / s')), -127, 127)
//   earlier rows, when s' > s:  code' = rint(code * (s / s'))
// A value that is not finite gives the page's scale the value NaN, so that
// attention over the page is NaN as it would be over the value itself.
#include <cuda_bf16.h>

#include "cache.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 128;

// 8 consecutive bf16 as floats
__device__ __forceinline__ void widen(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(u[e] << 16);
    x[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
  }
}

// Rotates the 8 values of columns [col, col + 8) of a row; `other` holds the
// columns half a rotation away (the pairing (i, i + dim / 2)).
__device__ __forceinline__ void rotate(const RopeRef& rope, int pos, int col, const float (&other)[8], float (&x)[8]) {
  const int half = rope.dim / 2;
  if (rope.interleaved) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(rope.cos + (size_t)pos * half + col / 2));
    const float4 s = __ldg(reinterpret_cast<const float4*>(rope.sin + (size_t)pos * half + col / 2));
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = x[2 * e], b = x[2 * e + 1];
      x[2 * e] = __fsub_rn(__fmul_rn(a, cc[e]), __fmul_rn(b, ss[e]));
      x[2 * e + 1] = __fadd_rn(__fmul_rn(b, cc[e]), __fmul_rn(a, ss[e]));
    }
  } else {
    const bool low = col < half;
    const int at = low ? col : col - half;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(rope.cos + (size_t)pos * half + at) + q);
      const float4 s = __ldg(reinterpret_cast<const float4*>(rope.sin + (size_t)pos * half + at) + q);
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float mine = x[4 * q + e], far = other[4 * q + e];
        x[4 * q + e] = low ? __fsub_rn(__fmul_rn(mine, cc[e]), __fmul_rn(far, ss[e]))
                           : __fadd_rn(__fmul_rn(mine, cc[e]), __fmul_rn(far, ss[e]));
      }
    }
  }
}

// grid (pieces, H, 2): one block quantises one page's new rows of one head of
// K (z = 0) or V (z = 1).  d / 8 lanes per row with 16 bytes each, the whole
// page in registers, all loads issued before the arithmetic: HBM-bound.
template <int D>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes, kPasses = kBlock / kRows;
  __shared__ uint32_t warp_max[kThreads / 32];
  const Piece pc = find_piece<kThreads>(p.b, (int)blockIdx.x, p.status);
  if (pc.b < 0) return;
  const int page = page_id(p.c, p.b, pc.b, pc.page_no, p.status);
  if (page < 0) return;
  const int tid = threadIdx.x, h = blockIdx.y;
  const bool is_k = blockIdx.z == 0;
  const int col = tid % kLanes * 8, r0 = tid / kLanes;
  const int rows = pc.hi - pc.lo;
  const uint16_t* src = is_k ? p.k + h * p.k_head : p.v + h * p.v_head;
  const long long pitch = is_k ? p.k_row : p.v_row;
  const bool turn = is_k && p.rope.cos != nullptr && col < p.rope.dim;
  const int half = p.rope.dim / 2;
  float* scale = (is_k ? p.c.k_scale : p.c.v_scale) + (size_t)page * p.c.H + h;
  int8_t* codes = (is_k ? p.c.k : p.c.v) + ((size_t)page * p.c.H + h) * kBlock * D;

  if (is_k && h == 0 && p.c.times != nullptr)
    for (int r = tid; r < rows; r += kThreads)
      p.c.times[(size_t)page * kBlock + pc.held + r] = p.row_times != nullptr ? p.row_times[pc.row + r] : NAN;

  uint4 w[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = r0 + i * kRows;
    w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows) w[i] = __ldg(reinterpret_cast<const uint4*>(src + (pc.row + r) * pitch + col));
  }
  const float s_old = pc.held > 0 ? *scale : 0.0f;

  auto value = [&](int i, int r, float (&x)[8]) {
    widen(w[i], x);
    if (turn && r < rows) {
      const int t = pc.row + r;
      int pos = p.rope.index != nullptr ? __ldg(p.rope.index + t) : pc.lo + r;
      if (pos < 0 || pos >= p.rope.n_pos) {
        cache_report(p.status, kStatusData);
        pos = min(max(pos, 0), p.rope.n_pos - 1);
      }
      float other[8];
      if (!p.rope.interleaved)
        widen(__ldg(reinterpret_cast<const uint4*>(src + t * pitch + (col < half ? col + half : col - half))), other);
      rotate(p.rope, pos, col, other, x);
    }
  };

  // |y| orders like its bit pattern, with infinity and NaN on top
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    float x[8];
    value(i, r0 + i * kRows, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if ((tid & 31) == 0) warp_max[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) top = max(top, warp_max[i]);

  float s_new;
  const bool bad = top >= 0x7F800000u || !(s_old <= 3.4e38f);
  if (bad) s_new = NAN;
  else s_new = fmaxf(fmaxf(s_old, __fdiv_rn(__uint_as_float(top), 127.0f)), kMinScale);
  const float inv = bad ? 0.0f : __frcp_rn(s_new);

#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = r0 + i * kRows;
    if (r >= rows) continue;
    float x[8];
    value(i, r, x);
    uint32_t c[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = bad ? 0.0f : __fmul_rn(x[e], inv);
      const int q = min(max(__float2int_rn(y), -127), 127);
      c[e >> 2] |= (uint32_t)(q & 0xFF) << (8 * (e & 3));
    }
    *reinterpret_cast<uint2*>(codes + (pc.held + r) * D + col) = make_uint2(c[0], c[1]);
  }
  if (pc.held > 0 && !bad && s_new > s_old) {
    const float ratio = __fdiv_rn(s_old, s_new);
    for (int i = tid; i < pc.held * (D / 4); i += kThreads) {
      uint32_t* at = reinterpret_cast<uint32_t*>(codes) + i;
      const uint32_t old = *at;
      uint32_t c = 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = (float)(int8_t)(old >> (8 * e));
        c |= (uint32_t)(__float2int_rn(__fmul_rn(x, ratio)) & 0xFF) << (8 * e);
      }
      *at = c;
    }
  }
  if (tid == 0) *scale = s_new;
}

// grid (pieces, H, 2): one block widens one page's rows of one head of K or V
// to bf16(code * scale); 16 codes per thread and step.
template <int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadParams p) {
  const Piece pc = find_piece<kThreads>(p.b, (int)blockIdx.x, p.status);
  if (pc.b < 0) return;
  const int page = page_id(p.c, p.b, pc.b, pc.page_no, p.status);
  const int h = blockIdx.y;
  const bool is_k = p.k != nullptr && blockIdx.z == 0;
  uint16_t* dst = (is_k ? p.k : p.v) + ((size_t)h * p.b.T + pc.row) * D;
  const size_t at = ((size_t)max(page, 0) * p.c.H + h);
  const float scale = page < 0 ? 0.0f : __ldg((is_k ? p.c.k_scale : p.c.v_scale) + at);
  const int8_t* codes = (is_k ? p.c.k : p.c.v) + at * kBlock * D + (size_t)pc.held * D;
  const int n = (pc.hi - pc.lo) * D / 16;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint4 w = page < 0 ? make_uint4(0u, 0u, 0u, 0u) : __ldg(reinterpret_cast<const uint4*>(codes) + i);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t x = u[e >> 1] >> (16 * (e & 1));
      const __nv_bfloat162 y = __floats2bfloat162_rn(__fmul_rn((float)(int8_t)x, scale),
                                                     __fmul_rn((float)(int8_t)(x >> 8), scale));
      o[e] = *reinterpret_cast<const uint32_t*>(&y);
    }
    uint4* to = reinterpret_cast<uint4*>(dst) + 2 * (size_t)i;
    to[0] = make_uint4(o[0], o[1], o[2], o[3]);
    to[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace

cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t stream) {
  const dim3 grid(max_pieces(p.b), (unsigned)p.c.H, 2);
  if (p.c.d == 64) append_kernel<64><<<grid, kThreads, 0, stream>>>(p);
  else append_kernel<128><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const ReadParams& p, cudaStream_t stream) {
  const dim3 grid(max_pieces(p.b), (unsigned)p.c.H, p.k != nullptr && p.v != nullptr ? 2 : 1);
  if (p.c.d == 64) read_kernel<64><<<grid, kThreads, 0, stream>>>(p);
  else read_kernel<128><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace h3
