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

#include <algorithm>

#include "cache.cuh"
#include "fastmath.cuh"
#include "ptx.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 256;
constexpr int kStages = 2;
constexpr int kBlocksPerSm = 3;

// 8 consecutive bf16 as four pairs of floats
__device__ __forceinline__ void widen(const uint4& w, uint64_t (&x)[4]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = f2_pack(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xFFFF0000u));
}

// One page's rotation table rows, as the block's rows use them.
struct Table {
  float cos[kBlock][64], sin[kBlock][64];
};

// Two products, each rounded.  A packed product that feeds a packed sum is
// otherwise fused into one rounding (also when both are written .rn), so it is
// taken as fma(a, b, -0) with a -0 that the compiler does not know.
__device__ __forceinline__ uint64_t mul2_rn(uint64_t a, uint64_t b, float minus_zero) {
  return f2_fma(a, b, f2_pack(minus_zero, minus_zero));
}

// the larger of a, |b| and |c|; NaN if one of them is
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return d;
}

// rint of two pairs, as bytes, for magnitudes below 2^22: adding 1.5 2^23
// rounds to an integer (ties to even) and leaves it in the low bits.
__device__ __forceinline__ uint32_t round4(uint64_t ab, uint64_t cd) {
  const uint64_t magic = f2_pack(12582912.0f, 12582912.0f);
  float a, b, c, d;
  f2_unpack(f2_add(ab, magic), a, b);
  f2_unpack(f2_add(cd, magic), c, d);
  return __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040),
                     __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040), 0x5410);
}

// Rotates the 8 values of columns [col, col + 8) of row r, two at a time (the
// packed operations round each half as the single ones do); `far` holds the
// columns half a rotation away (the pairing (i, i + dim / 2)), negated for the
// lower half, so that both halves add.
__device__ __forceinline__ void rotate(const Table& tab, const RopeRef& rope, int r, int col, const uint64_t (&far)[4],
                                       uint64_t (&x)[4], float mz) {
  if (rope.interleaved) {
    const float4 c = *reinterpret_cast<const float4*>(&tab.cos[r][col / 2]);
    const float4 s = *reinterpret_cast<const float4*>(&tab.sin[r][col / 2]);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a, b;
      f2_unpack(x[e], a, b);
      x[e] = f2_add(mul2_rn(x[e], f2_pack(cc[e], cc[e]), mz), mul2_rn(f2_pack(b, a), f2_pack(-ss[e], ss[e]), mz));
    }
  } else {
    const int half = rope.dim / 2, at = col < half ? col : col - half;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float4 c = *reinterpret_cast<const float4*>(&tab.cos[r][at + 4 * q]);
      const float4 s = *reinterpret_cast<const float4*>(&tab.sin[r][at + 4 * q]);
      const uint64_t c2[2] = {f2_pack(c.x, c.y), f2_pack(c.z, c.w)}, s2[2] = {f2_pack(s.x, s.y), f2_pack(s.z, s.w)};
#pragma unroll
      for (int e = 0; e < 2; ++e)
        x[2 * q + e] = f2_add(mul2_rn(x[2 * q + e], c2[e], mz), mul2_rn(far[2 * q + e], s2[e], mz));
    }
  }
}

// grid (pieces, ceil(2 H / per)): one block quantises one page's new rows of
// `per` of the 2 H heads of K and V, one after the other.  HBM-bound: d / 8 lanes
// per row with 16 bytes each, brought by cp.async kStages - 1 heads ahead into a
// ring whose rows only their own warp touches; the rotation table's rows are in
// shared memory for all heads.  Finding the piece, its page and its table rows
// takes about as long as two heads, so a large call gives a block many.
// Measured: 16,384 rows of 56 heads of 128 with rotation 169 us (705 MB, 4.2 TB/s;
// what is left is issue: about 400 instructions per warp and head).
template <int D>
struct AppendLayout {
  static constexpr int kStage = kBlock * D * 2;
  static constexpr int kBytes = kStages * kStage + (int)sizeof(Table);
};
template <int D>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) append_kernel(const AppendParams p, int per) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes, kPasses = kBlock / kRows;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) uint32_t warp_max[2][kThreads / 32];
  __shared__ Piece piece;
  const Table& tab = *reinterpret_cast<const Table*>(smem + kStages * AppendLayout<D>::kStage);
  Table& tab_w = *reinterpret_cast<Table*>(smem + kStages * AppendLayout<D>::kStage);
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < 32) {
    const Piece x = find_piece(p.b, (int)blockIdx.x, p.status);
    if (tid == 0) piece = x;
  }
  __syncthreads();
  const Piece pc = piece;
  if (pc.b < 0) return;
  const int t0 = blockIdx.y * per, t1 = min(2 * p.c.H, t0 + per);  // task t: head t of K, or t - H of V
  const int col = tid % kLanes * 8, r0 = tid / kLanes;
  const int rows = pc.hi - pc.lo;
  const bool turns = p.rope.cos != nullptr;
  const int half = p.rope.dim / 2;
  const uint32_t ring = smem_u32(smem) + (uint32_t)(r0 * D + col) * 2;

  auto issue = [&](int t) {
    if (t < t1) {
      const bool is_k = t < p.c.H;
      const long long pitch = is_k ? p.k_row : p.v_row;
      const uint16_t* src =
          (is_k ? p.k + t * p.k_head : p.v + (t - p.c.H) * p.v_head) + (pc.row + r0) * pitch + col;
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
        if (r0 + i * kRows < rows)
          cp_async16(ring + (uint32_t)(t % kStages * AppendLayout<D>::kStage + i * kRows * D * 2), src + i * kRows * pitch);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int t = 0; t < kStages - 1; ++t) issue(t0 + t);
  const int page = page_id(p.c, p.b, pc.b, pc.page_no, p.status);
  if (t0 == 0 && page >= 0 && p.c.times != nullptr)
    for (int r = tid; r < rows; r += kThreads)
      p.c.times[(size_t)page * kBlock + pc.held + r] = p.row_times != nullptr ? p.row_times[pc.row + r] : NAN;
  if (turns && t0 < p.c.H) {
    const int quads = half / 4;  // 16-byte pieces of a table row
    for (int i = tid; i < rows * quads; i += kThreads) {
      const int r = i / quads, q = i % quads;
      int pos = p.rope.index != nullptr ? __ldg(p.rope.index + pc.row + r) : pc.lo + r;
      if (pos < 0 || pos >= p.rope.n_pos) {
        report(p.status, kStatusData);
        pos = min(max(pos, 0), p.rope.n_pos - 1);
      }
      reinterpret_cast<float4*>(tab_w.cos[r])[q] = __ldg(reinterpret_cast<const float4*>(p.rope.cos + (size_t)pos * half) + q);
      reinterpret_cast<float4*>(tab_w.sin[r])[q] = __ldg(reinterpret_cast<const float4*>(p.rope.sin + (size_t)pos * half) + q);
    }
  }
  __syncthreads();
  if (page < 0) {
    cp_async_wait<0>();
    return;
  }

  for (int t = t0; t < t1; ++t) {
    const bool is_k = t < p.c.H, turn = is_k && turns;
    const size_t at = (size_t)page * p.c.H + (is_k ? t : t - p.c.H);
    float* scale = (is_k ? p.c.k_scale : p.c.v_scale) + at;
    int8_t* codes = (is_k ? p.c.k : p.c.v) + at * kBlock * D;
    const float s_old = pc.held > 0 ? *scale : 0.0f;
    cp_async_wait<kStages - 2>();
    __syncwarp();  // the warp's rows of this stage have landed, and the stage issued next is read
    const uint8_t* mine = smem + t % kStages * AppendLayout<D>::kStage + (r0 * D + col) * 2;
    issue(t + kStages - 1);
    uint64_t y[kPasses][4];
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = r0 + i * kRows;
      const uint8_t* src = mine + i * kRows * D * 2;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) w = *reinterpret_cast<const uint4*>(src);
      widen(w, y[i]);
      if (turn && r < rows && col < p.rope.dim) {
        uint64_t far[4];
        if (!p.rope.interleaved) {
          const uint32_t sign = col < half ? 0x80008000u : 0u;
          const uint4 v = *reinterpret_cast<const uint4*>(col < half ? src + half * 2 : src - half * 2);
          widen(make_uint4(v.x ^ sign, v.y ^ sign, v.z ^ sign, v.w ^ sign), far);
        }
        rotate(tab, p.rope, r, col, far, y[i], p.minus_zero);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a, b;
        f2_unpack(y[i][e], a, b);
        most = max_abs_nan(most, a, b);
      }
    }
    // magnitudes order like their bit patterns, with infinity and NaN on top
    uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most) & 0x7FFFFFFFu);
    uint32_t* wm = warp_max[t & 1];  // two sets: one barrier per task is enough
    if (lane == 0) wm[tid >> 5] = top;
    __syncthreads();
    const uint4 wa = *reinterpret_cast<const uint4*>(wm), wb = *reinterpret_cast<const uint4*>(wm + 4);
    top = max(max(max(wa.x, wa.y), max(wa.z, wa.w)), max(max(wb.x, wb.y), max(wb.z, wb.w)));

    const bool bad = top >= 0x7F800000u || !(s_old <= 3.4e38f);
    const float s_new = bad ? NAN : fmaxf(fmaxf(s_old, __fdiv_rn(__uint_as_float(top), 127.0f)), kMinScale);
    const float inv = bad ? 0.0f : __frcp_rn(s_new);
    const uint64_t inv2 = f2_pack(inv, inv);
    int8_t* dst = codes + (pc.held + r0) * D + col;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = r0 + i * kRows;
      if (r >= rows) continue;
      // |y| / s' <= 127 up to roundings far below a half, so the clamp has nothing to do
      uint2 c = make_uint2(0u, 0u);
      if (!bad)
        c = make_uint2(round4(mul2_rn(y[i][0], inv2, p.minus_zero), mul2_rn(y[i][1], inv2, p.minus_zero)),
                       round4(mul2_rn(y[i][2], inv2, p.minus_zero), mul2_rn(y[i][3], inv2, p.minus_zero)));
      *reinterpret_cast<uint2*>(dst + i * kRows * D) = c;
    }
    if (pc.held > 0 && !bad && s_new > s_old) {
      const float ratio = __fdiv_rn(s_old, s_new);
      for (int i = tid; i < pc.held * (D / 4); i += kThreads) {
        uint32_t* old = reinterpret_cast<uint32_t*>(codes) + i;
        const uint32_t c = *old;
        const uint64_t ratio2 = f2_pack(ratio, ratio);
        *old = round4(mul2_rn(f2_pack((float)(int8_t)c, (float)(int8_t)(c >> 8)), ratio2, p.minus_zero),
                      mul2_rn(f2_pack((float)(int8_t)(c >> 16), (float)(int8_t)(c >> 24)), ratio2, p.minus_zero));
      }
    }
    if (tid == 0) *scale = s_new;
  }
}

// grid (pieces, H, 2): one block widens one page's rows of one head of K or V
// to bf16(code * scale), 16 codes per load, all of a thread's loads issued
// first.  HBM-bound: 16,384 rows of 56 heads of 128 in 127 us (5.6 TB/s).
template <int D>
__global__ void __launch_bounds__(128) read_kernel(const ReadParams p) {
  constexpr int kLoads = kBlock * D / 16 / 128;
  const Piece pc = find_piece(p.b, (int)blockIdx.x, p.status);
  if (pc.b < 0) return;
  const int page = page_id(p.c, p.b, pc.b, pc.page_no, p.status);
  const int h = blockIdx.y;
  const bool is_k = p.k != nullptr && blockIdx.z == 0;
  const size_t at = (size_t)max(page, 0) * p.c.H + h;
  const int8_t* codes = (is_k ? p.c.k : p.c.v) + at * kBlock * D + (size_t)pc.held * D;
  const int n = (pc.hi - pc.lo) * D / 16;
  uint4 w[kLoads];
#pragma unroll
  for (int x = 0; x < kLoads; ++x) {
    const int i = threadIdx.x + x * 128;
    w[x] = make_uint4(0u, 0u, 0u, 0u);
    if (page >= 0 && i < n) w[x] = __ldg(reinterpret_cast<const uint4*>(codes) + i);
  }
  const float scale = page < 0 ? 0.0f : __ldg((is_k ? p.c.k_scale : p.c.v_scale) + at);
  uint4* dst = reinterpret_cast<uint4*>((is_k ? p.k : p.v) + ((size_t)h * p.b.T + pc.row) * D);
#pragma unroll
  for (int x = 0; x < kLoads; ++x) {
    const int i = threadIdx.x + x * 128;
    if (i >= n) break;
    const uint32_t u[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t c = u[e >> 1] >> (16 * (e & 1));
      const __nv_bfloat162 y = __floats2bfloat162_rn(__fmul_rn((float)(int8_t)c, scale),
                                                     __fmul_rn((float)(int8_t)(c >> 8), scale));
      o[e] = *reinterpret_cast<const uint32_t*>(&y);
    }
    dst[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace

namespace {
template <int D>
cudaError_t launch_append_t(const AppendParams& p, cudaStream_t stream) {
  constexpr int bytes = AppendLayout<D>::kBytes;
  const cudaError_t e = cudaFuncSetAttribute(append_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  // As many heads per block as leave one wave of blocks, 16 at most: 16,384 rows of
  // 56 heads take 169 us with 16, 292 us with 1; 3,400 rows of 24 heads of 64 17 us
  // with 7, 31 us with 1; a token of eight sequences has one head per block.
  const unsigned pieces = max_pieces(p.b);
  const int per = (int)std::min(16ll, std::max(1ll, (long long)pieces * 2 * p.c.H / (148 * kBlocksPerSm)));
  append_kernel<D><<<dim3(pieces, (unsigned)((2 * p.c.H + per - 1) / per)), kThreads, bytes, stream>>>(p, per);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t stream) {
  return p.c.d == 64 ? launch_append_t<64>(p, stream) : launch_append_t<128>(p, stream);
}

cudaError_t launch_cache_read(const ReadParams& p, cudaStream_t stream) {
  const dim3 grid(max_pieces(p.b), (unsigned)p.c.H, p.k != nullptr && p.v != nullptr ? 2 : 1);
  if (p.c.d == 64) read_kernel<64><<<grid, 128, 0, stream>>>(p);
  else read_kernel<128><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace h3
