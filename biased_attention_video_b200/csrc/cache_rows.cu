// Attention over the paged int8 cache for few query rows per sequence (one
// token, a handful of drafts): per query row i of sequence b and head h, over
// the cached rows j < length[b] (causal: j <= length[b] - rows + i)
//   s_j = (q . code_j) s_k / sqrt(d) - penalty(|t_q - t_j|),
//   O = sum_j exp(s_j) code_j s_v / sum_j exp(s_j),   LSE = log sum_j exp(s_j);
// a row that sees no key gets O = 0 and LSE = -inf.
//
// HBM-bound: every code is read once and used for the few rows of one sequence
// and K/V head.  The query heads of a K/V head and the rows of a sequence form
// one list of (row, head) pairs, cut into tiles of 8 NT pairs; an item is one
// tile of one sequence and K/V head, its units are the sequence's pages.  The
// units of all items form one line that the blocks share evenly, whatever the
// lengths are (they are read on the device); a block walks its stretch item by
// item, and items that lie in several blocks are joined by a second launch from
// partial results (maximum, sum, unnormalised O in fp32).
//
// Inside a block each warp streams granules of 16 keys on its own: cp.async into
// a ring of its own (no barrier between warps until the item ends), then
//   S^T = K Q^T   mma m16n8k16 fp16, A = the codes widened exactly to fp16,
//   P^T           exp2 of the scaled scores, packed to fp16, transposed by movmatrix,
//   O^T += V^T P^T  A = the V codes, two keys of a column per register.
// fp16 and not bf16 operands, for a code widens to fp16 in two operations for
// two codes instead of three and the kernel is near the instruction rate: Q is
// scaled per row by a power of two to a maximum in [2^9, 2^10) (its 8-bit
// mantissas stay exact down to 2^-23 of the row's maximum), and the V scale goes
// into the exponent, so that a probability times its V scale is 2^12 at the row's
// largest and keeps more bits than bf16 would down to 2^-26 of that.
// The d order of A and of Q agree by construction and nothing else sees it, so
// a lane takes 16 consecutive bytes of a row per load.  mma.sync and not tcgen05:
// 8 rows fill no 128-row tile, and the widened codes are in registers anyway.
#include <cuda_bf16.h>

#include <type_traits>

#include "cache_attn.cuh"

namespace h3 {
namespace {

using namespace sm;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kKeys = 16;    // keys of a granule
constexpr int kStages = 3;
constexpr int kJoinWarps = 16;
constexpr float kRaise = 3.0f;   // log2 units: a score this far above the running maximum raises it
constexpr float kShift = 12.0f;  // a probability is 2^kShift at the running maximum: at most 2^15 in fp16
constexpr int kBlocksPerSm = 2;
constexpr int kGrid = 148 * kBlocksPerSm;
constexpr int kMinShare = kWarps * kKeys / kBlock;  // pages: one granule for every warp

template <int D, int NT>
struct RowsLayout {
  static constexpr int kRows = 8 * NT;
  static constexpr int kV = kKeys * D;              // V codes after the K codes
  static constexpr int kMeta = 2 * kKeys * D;       // k scale, v scale, valid keys, -, then the keys' times
  static constexpr int kStage = kMeta + 16 + kKeys * 4;
  static constexpr int kPitch = D + 4;              // floats of one row of the warps' results
  static constexpr int kResult = kRows * kPitch * 4;
  static constexpr int kRing = kStages * kStage > kResult ? kStages * kStage : kResult;
  static constexpr int kQ = kWarps * kRing;         // Q fragments: [D / 16][NT][32] uint2
  static constexpr int kQScale = kQ + D / 16 * NT * 256;  // [R] powers of two
  static constexpr int kMl = kQScale + kRows * 4;
  static constexpr int kBytes = kMl + kWarps * kRows * 8;
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// The codes in bytes 0 and 2 of w as two fp16: with 0x64 in front, a byte with its
// sign bit flipped reads as 1024 + (128 + code).
__device__ __forceinline__ uint32_t widen2h(uint32_t w) {
  uint32_t x, r;
  asm("lop3.b32 %0, %1, 0x00FF00FF, 0x64806480, 0x6A;" : "=r"(x) : "r"(w));  // (w & a) ^ b
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x64806480u));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// ---------------------------------------------------------------- the line

// Sequence b's share of the line: tiles x K/V heads x pages (at least one page,
// so that a sequence without cached rows still gets its rows written).
struct Seq {
  int first, n, len, pages;
  long long tiles, units;
};
template <int R>
__device__ __forceinline__ Seq load_seq(const CacheAttnParams& p, int b) {
  Seq s;
  const SeqRows r = seq_rows(p.b, b, p.status);
  s.first = r.first;
  s.n = r.n;
  s.len = seq_length(p.b, b, p.status);
  s.pages = max(1, (s.len + kBlock - 1) / kBlock);
  s.tiles = ((long long)s.n * p.group + R - 1) / R;
  s.units = s.tiles * p.c.H * s.pages;
  return s;
}

__device__ __forceinline__ long long scan_warp(long long v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long w = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += w;
  }
  return v;
}

// The line, known to a block of NT threads.  Up to NT sequences are scanned once
// and a thread keeps its sequence's place; more are gone through in rounds.
template <int R, int NT>
struct Line {
  long long total, lo, mine;  // lo, mine: of sequence threadIdx.x, for B <= NT
  __device__ __forceinline__ explicit Line(const CacheAttnParams& p) {
    __shared__ long long sums[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    mine = 0;
    for (int b = tid; b < p.b.B; b += NT) mine += load_seq<R>(p, b).units;
    const long long incl = scan_warp(mine);
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    total = 0;
    lo = incl - mine;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) lo += sums[w];
      total += sums[w];
    }
  }
  // The sequence that unit u lies in, and the line before that sequence.
  __device__ __forceinline__ int find(const CacheAttnParams& p, long long u, long long* before) const {
    __shared__ long long sums[NT / 32], at;
    __shared__ int found;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (p.b.B <= NT) {
      if (u >= lo && u < lo + mine) {
        found = tid;
        at = lo;
      }
    } else {
      long long base = 0;
      for (int b0 = 0; b0 < p.b.B && base <= u; b0 += NT) {
        const long long units = b0 + tid < p.b.B ? load_seq<R>(p, b0 + tid).units : 0;
        const long long incl = scan_warp(units);
        __syncthreads();
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        long long from = base + incl - units;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
          if (w < warp) from += sums[w];
          base += sums[w];
        }
        if (u >= from && u < from + units) {
          found = b0 + tid;
          at = from;
        }
      }
    }
    __syncthreads();
    *before = at;
    return found;
  }
};

__device__ __forceinline__ long long share_of(long long total) {
  const long long even = (total + kGrid - 1) / kGrid;
  return even > kMinShare ? even : kMinShare;
}

// Output row (head T + packed row) of a pair of the sequence's list.
__device__ __forceinline__ size_t row_of(const CacheAttnParams& p, const Seq& s, int hk, long long pair) {
  return (size_t)(hk * p.group + (int)(pair % p.group)) * p.b.T + s.first + (int)(pair / p.group);
}

// Slot of partial results: unnormalised O [R][D], then (maximum, sum) [R].
// Block c's slot 0 holds an item that an earlier block began, slot 1 the item
// that it begins and a later one goes on with.
template <int D, int R>
__device__ __forceinline__ float* slot_of(const CacheAttnParams& p, long long block, int which) {
  return p.partial + (2 * block + which) * (size_t)(R * (D + 2));
}

// --------------------------------------------------------------- the kernel

template <int D, int NT, bool kPen>
__global__ void __launch_bounds__(kThreads, NT > 2 ? 1 : kBlocksPerSm) rows_kernel(const CacheAttnParams p) {
  using L = RowsLayout<D, NT>;
  constexpr int R = L::kRows, kJ = D / 16;
  constexpr bool kQRegs = NT == 1;  // Q fragments in registers, else read from shared memory
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * L::kRing;
  const uint32_t ring_a = smem_u32(ring), q_a = smem_u32(smem + L::kQ);
  float2* ml = reinterpret_cast<float2*>(smem + L::kMl);  // [warp][R] (maximum, sum)

  launch_dependents();
  const Line<R, kThreads> line(p);
  const long long total = line.total, share = share_of(total);
  const long long u0 = blockIdx.x * share, u1 = min(total, u0 + share);
  if (u0 >= u1) return;
  long long before;
  int b = line.find(p, u0, &before);
  Seq s = load_seq<R>(p, b);

  for (long long u = u0; u < u1;) {
    while (u >= before + s.units) {
      before += s.units;
      s = load_seq<R>(p, ++b);
    }
    // item: tile by tile, K/V head by K/V head, page by page
    const long long item = (u - before) / s.pages, item_u = before + item * s.pages;
    const int hk = (int)(item % p.c.H);
    const long long pair0 = item / p.c.H * R;
    const int page0 = (int)(u - item_u), page1 = (int)min((long long)s.pages, u1 - item_u);
    const int pairs = (int)min((long long)R, (long long)s.n * p.group - pair0);

    // Q fragments of the item (8 columns n = pairs; k = the columns of a word of codes)
    __syncthreads();  // the last item's results and fragments are read
    uint32_t qf[kQRegs ? 2 * kJ : 1];
    if (kQRegs || warp < NT) {
      const int r = (kQRegs ? 0 : warp * 8) + g;
      const uint16_t* src = nullptr;
      if (r < pairs) {
        const long long pair = pair0 + r;
        const int h = hk * p.group + (int)(pair % p.group);
        src = p.q + h * p.q_head + (s.first + pair / p.group) * p.q_row;
      }
      float y[D / 4], top = 0.0f;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint4 w[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (src != nullptr) {
          w[0] = __ldg(reinterpret_cast<const uint4*>(src + c * 64 + t * 16));
          w[1] = __ldg(reinterpret_cast<const uint4*>(src + c * 64 + t * 16) + 1);
        }
        const uint32_t x[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[16 * c + 2 * i] = __uint_as_float(x[i] << 16);
          y[16 * c + 2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
          top = fmaxf(top, fmaxf(fabsf(y[16 * c + 2 * i]), fabsf(y[16 * c + 2 * i + 1])));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
      // 2^(9 - exponent of the row's maximum); a row of zeros or with an infinity stays as it is
      int e = (int)(__float_as_uint(top) >> 23) - 127;
      e = top == 0.0f || e > 127 ? 9 : max(e, -110);
      const float up = __uint_as_float((uint32_t)(127 + 9 - e) << 23);
      if (t == 0) reinterpret_cast<float*>(smem + L::kQScale)[r] = __uint_as_float((uint32_t)(127 + e - 9) << 23);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {  // word i: codes 4 i .. 4 i + 3, in the order (0, 2), (1, 3)
        const uint32_t f0 = pack_f16(y[4 * i] * up, y[4 * i + 2] * up);
        const uint32_t f1 = pack_f16(y[4 * i + 1] * up, y[4 * i + 3] * up);
        if constexpr (kQRegs) {
          qf[2 * i] = f0;
          qf[2 * i + 1] = f1;
        } else {
          reinterpret_cast<uint2*>(smem + L::kQ)[(i * NT + warp) * 32 + lane] = make_uint2(f0, f1);
        }
      }
    }
    __syncthreads();
    // what this lane's pairs may see, and their times
    int lim[NT][2], lim_all = s.len;
    float tq[NT][2], qs[NT][2];
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * x + 2 * t + e;
        lim[x][e] = s.len;
        tq[x][e] = NAN;
        qs[x][e] = reinterpret_cast<const float*>(smem + L::kQScale)[r] * p.scale_log2;
        if (r < pairs) {
          const int i = (int)((pair0 + r) / p.group);
          if (p.causal) lim[x][e] = min(s.len, max(0, s.len - s.n + i + 1));
          if (kPen) tq[x][e] = __ldg(p.q_times + s.first + i);
        }
        lim_all = min(lim_all, lim[x][e]);
      }
    lim_all = __reduce_min_sync(kFull, lim_all);

    float o[NT][kJ][4] = {}, m[NT][2], l[NT][2] = {};
#pragma unroll
    for (int x = 0; x < NT; ++x) m[x][0] = m[x][1] = -INFINITY;

    const int end = min(s.len, page1 * kBlock);
    const int first = page0 * kBlock + warp * kKeys;  // keys first, first + kWarps * kKeys, ...
    const int steps = first < end ? (end - first + kWarps * kKeys - 1) / (kWarps * kKeys) : 0;

    auto issue = [&](int i) {
      if (i < steps) {
        const int key = first + i * (kWarps * kKeys);
        const int page = page_id(p.c, p.b, b, key / kBlock, p.status);
        const uint32_t st = ring_a + i % kStages * L::kStage;
        if (page >= 0) {
          const size_t at = (size_t)page * p.c.H + hk;
          const size_t off = at * kBlock * D + (size_t)(key % kBlock) * D;
#pragma unroll
          for (int c = 0; c < kKeys * D / 512; ++c) {
            const int idx = c * 32 + lane, row = idx / (D / 16), ch = idx % (D / 16);
            const int ck = D == 128 ? ch ^ ((row & 1) << 2) : ch;
            const int cv = D == 128 ? ch ^ ((row >> 1 & 3) << 1) : ch ^ (row >> 1 & 3);
            cp_async16(st + row * D + ck * 16, p.c.k + off + idx * 16);
            cp_async16(st + L::kV + row * D + cv * 16, p.c.v + off + idx * 16);
          }
          if (lane == 0) cp_async4(st + L::kMeta, p.c.k_scale + at);
          if (lane == 1) cp_async4(st + L::kMeta + 4, p.c.v_scale + at);
          if (kPen && lane >= 8 && lane < 8 + kKeys / 4)
            cp_async16(st + L::kMeta + 16 + (lane - 8) * 16,
                       p.c.times + (size_t)page * kBlock + key % kBlock + (lane - 8) * 4);
        }
        if (lane == 2)
          *reinterpret_cast<int*>(ring + i % kStages * L::kStage + L::kMeta + 8) = page >= 0 ? min(kKeys, end - key) : 0;
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    for (int i = 0; i < steps; ++i) {
      cp_async_wait<kStages - 2>();
      __syncwarp();  // every lane's copies of this stage have landed, and the stage issued next is read
      issue(i + kStages - 1);
      const uint32_t st = ring_a + i % kStages * L::kStage;
      const float* meta = reinterpret_cast<const float*>(ring + i % kStages * L::kStage + L::kMeta);
      const int live = __float_as_int(meta[2]);
      if (live == 0) continue;
      // a V scale that is not finite marks the probabilities of the keys that are seen, and only those
      const float ks = meta[0], vs = meta[1], lv = log2_approx(vs), iv = vs < 3.0e38f ? rcp_approx(vs) : 1.0f;
      const int key = first + i * (kWarps * kKeys);

      // S^T: 16 keys x 8 NT pairs
      float acc[NT][4] = {};
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const int ch = D == 128 ? (4 * c + t) ^ ((g & 1) << 2) : t;
        const uint4 wa = lds128(st + g * D + ch * 16), wb = lds128(st + (g + 8) * D + ch * 16);
        const uint32_t ra[4] = {wa.x, wa.y, wa.z, wa.w}, rb[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t a0 = widen2h(ra[w]), a1 = widen2h(rb[w]), a2 = widen2h(ra[w] >> 8), a3 = widen2h(rb[w] >> 8);
#pragma unroll
          for (int x = 0; x < NT; ++x) {
            uint2 f;
            if constexpr (kQRegs) f = make_uint2(qf[2 * (4 * c + w)], qf[2 * (4 * c + w) + 1]);
            else f = lds64(q_a + (((4 * c + w) * NT + x) * 32 + lane) * 8);
            mma_f16(acc[x], a0, a1, a2, a3, f.x, f.y);
          }
        }
      }
      // scores times V scales in log2 units: [x][0], [x][1] key g, [x][2], [x][3] key g + 8
      float over = -1.0f;  // whether one lies kRaise above its pair's running maximum
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = fmaf(acc[x][e], qs[x][e & 1] * ks, lv);
          if (kPen) {
            const float ex = fmaxf(fabsf(tq[x][e & 1] - meta[4 + g + (e >> 1) * 8]) - p.window, 0.0f) * p.inv_falloff;
            v -= fminf(p.strength_log2 * ex * ex, p.cap_log2);
          }
          acc[x][e] = v;
        }
      if (key + live > lim_all || live < kKeys) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int kk = g + (e >> 1) * 8;
            if (kk >= live || key + kk >= lim[x][e & 1]) acc[x][e] = -INFINITY;
          }
      }
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        if (fmaxf(acc[x][0], acc[x][2]) > m[x][0] + kRaise) over = 1.0f;
        if (fmaxf(acc[x][1], acc[x][3]) > m[x][1] + kRaise) over = 1.0f;
      }
      if (__any_sync(kFull, over > 0.0f)) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(acc[x][e], acc[x][e + 2]);
#pragma unroll
            for (int q = 4; q < 32; q <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, q));
            const float mn = fmaxf(m[x][e], mx);
            const float alpha = m[x][e] == mn ? 1.0f : ex2(m[x][e] - mn);
            m[x][e] = mn;
            l[x][e] *= alpha;
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
              o[x][j][e] *= alpha;
              o[x][j][e + 2] *= alpha;
            }
          }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        const float m0 = (m[x][0] == -INFINITY ? 0.0f : m[x][0]) - kShift;
        const float m1 = (m[x][1] == -INFINITY ? 0.0f : m[x][1]) - kShift;
        const float p0 = ex2(acc[x][0] - m0), p1 = ex2(acc[x][1] - m1);
        const float p2 = ex2(acc[x][2] - m0), p3 = ex2(acc[x][3] - m1);
        l[x][0] = fmaf(p0 + p2, iv, l[x][0]);
        l[x][1] = fmaf(p1 + p3, iv, l[x][1]);
        pb[x][0] = transpose8x8(pack_f16(p0, p1));
        pb[x][1] = transpose8x8(pack_f16(p2, p3));
      }
      // O^T += V^T P^T: this lane's keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9, its columns from g D / 8 on
      uint32_t v[4][D / 32];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 2 * t + (r & 1) + (r >> 1) * 8;
        const uint32_t a = st + L::kV + row * D;
        if constexpr (D == 128) {
          const uint4 w = lds128(a + ((g ^ ((row >> 1 & 3) << 1)) << 4));
          v[r][0] = w.x, v[r][1] = w.y, v[r][2] = w.z, v[r][3] = w.w;
        } else {
          const uint2 w = lds64(a + (((g >> 1) ^ (row >> 1 & 3)) << 4) + (g & 1) * 8);
          v[r][0] = w.x, v[r][1] = w.y;
        }
      }
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const uint32_t sel = j & 1 ? 0x7632 : 0x5410;
        const uint32_t ab = __byte_perm(v[0][j >> 1], v[1][j >> 1], sel);
        const uint32_t cd = __byte_perm(v[2][j >> 1], v[3][j >> 1], sel);
        const uint32_t a0 = widen2h(ab), a1 = widen2h(ab >> 8), a2 = widen2h(cd), a3 = widen2h(cd >> 8);
#pragma unroll
        for (int x = 0; x < NT; ++x) mma_f16(o[x][j], a0, a1, a2, a3, pb[x][0], pb[x][1]);
      }
    }
    cp_async_wait<0>();
    __syncwarp();

    // the warps' results, over their own rings
    float* res = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * x + 2 * t + e;
#pragma unroll
        for (int q = 4; q < 32; q <<= 1) l[x][e] += __shfl_xor_sync(kFull, l[x][e], q);
        if (g == 0) ml[warp * R + r] = make_float2(m[x][e] - kShift, l[x][e]);
#pragma unroll
        for (int j = 0; j < kJ; ++j)
          *reinterpret_cast<float2*>(res + r * L::kPitch + g * (D / 8) + 2 * j) = make_float2(o[x][j][e], o[x][j][e + 2]);
      }
    __syncthreads();
    const bool whole = page0 == 0 && page1 == s.pages;
    float* slot = whole ? nullptr : slot_of<D, R>(p, blockIdx.x, page0 > 0 ? 0 : 1);
    for (int i = tid; i < R * (D / 4); i += kThreads) {
      const int r = i / (D / 4), col = i % (D / 4) * 4;
      if (r >= pairs) break;
      float mm = -INFINITY, ll = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ml[w * R + r].x);
      float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 x = ml[w * R + r];
        const float a = x.x == -INFINITY ? 0.0f : ex2(x.x - mm);
        const float4 y = *reinterpret_cast<const float4*>(smem + w * L::kRing + (r * L::kPitch + col) * 4);
        ll += a * x.y;
        sum.x += a * y.x, sum.y += a * y.y, sum.z += a * y.z, sum.w += a * y.w;
      }
      if (whole) {
        const size_t at = row_of(p, s, hk, pair0 + r);
        store_cols(p, at, col, sum, ll == 0.0f ? 0.0f : 1.0f / ll);
        if (col == 0) store_lse(p, at, mm, ll);
      } else {
        *reinterpret_cast<float4*>(slot + r * D + col) = sum;
        if (col == 0) *reinterpret_cast<float2*>(slot + R * D + 2 * r) = make_float2(mm, ll);
      }
    }
    u = item_u + page1;
  }
}

// Joins the items that several blocks share: block x looks at the border
// between the stretches x and x + 1 and joins the item that lies across it, if
// it is that item's first border.
//
// kWays warps share a pair's slots; a lane holds D / 32 columns.
template <int D, int NT>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const CacheAttnParams p) {
  constexpr int R = 8 * NT, kWays = kJoinWarps > R ? kJoinWarps / R : 1, kCols = D / 32;
  using Cols = typename std::conditional<kCols == 4, float4, float2>::type;
  __shared__ float part[kWays > 1 ? kJoinWarps : 1][D + 2];
  const Line<R, 32 * kJoinWarps> line(p);
  const long long total = line.total, share = share_of(total);
  const long long c0 = blockIdx.x, u = (c0 + 1) * share;
  if (u >= total) {
    wait_dependency();
    return;
  }
  long long before;
  const int b = line.find(p, u, &before);
  const Seq s = load_seq<R>(p, b);
  const long long item = (u - before) / s.pages, lo = before + item * s.pages, hi = lo + s.pages;
  wait_dependency();
  if (lo == u || lo / share != c0) return;
  const int n = (int)((hi - 1) / share - c0) + 1;  // slots
  const int hk = (int)(item % p.c.H);
  const long long pair0 = item / p.c.H * R;
  const int pairs = (int)min((long long)R, (long long)s.n * p.group - pair0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, way = warp % kWays;
  auto slot = [&](int c) { return slot_of<D, R>(p, c0 + c, c == 0 ? 1 : 0); };
  for (int r = warp / kWays; r < R; r += kJoinWarps / kWays) {
    float mm = -INFINITY, ll = 0.0f, sum[kCols] = {};
    if (r < pairs)
      for (int c = way; c < n; c += 32 * kWays) {  // 32 slots at a time, a lane for each
        const int mine = c + lane * kWays;
        const float2 x = mine < n ? *reinterpret_cast<const float2*>(slot(mine) + R * D + 2 * r)
                                  : make_float2(-INFINITY, 0.0f);
        float mn = fmaxf(mm, x.x);
#pragma unroll
        for (int q = 16; q > 0; q >>= 1) mn = fmaxf(mn, __shfl_xor_sync(kFull, mn, q));
        const float base = mn == -INFINITY ? 0.0f : mn, a = ex2(mm - base), w = ex2(x.x - base);
        float lw = w * x.y;
#pragma unroll
        for (int q = 16; q > 0; q >>= 1) lw += __shfl_xor_sync(kFull, lw, q);
        mm = mn;
        ll = ll * a + lw;
#pragma unroll
        for (int e = 0; e < kCols; ++e) sum[e] *= a;
        const int live = min(32, (n - c + kWays - 1) / kWays);
#pragma unroll 8
        for (int k = 0; k < live; ++k) {
          const float wk = __shfl_sync(kFull, w, k);
          const Cols y = *(reinterpret_cast<const Cols*>(slot(c + k * kWays) + r * D) + lane);
          const float* yy = reinterpret_cast<const float*>(&y);
#pragma unroll
          for (int e = 0; e < kCols; ++e) sum[e] = fmaf(wk, yy[e], sum[e]);
        }
      }
    if constexpr (kWays > 1) {
#pragma unroll
      for (int e = 0; e < kCols; ++e) part[warp][lane * kCols + e] = sum[e];
      if (lane == 0) part[warp][D] = mm, part[warp][D + 1] = ll;
      __syncthreads();
      if (way == 0) {
#pragma unroll
        for (int k = 1; k < kWays; ++k) {
          const float mk = part[warp + k][D], mn = fmaxf(mm, mk), base = mn == -INFINITY ? 0.0f : mn;
          const float a = ex2(mm - base), w = ex2(mk - base);
          mm = mn;
          ll = ll * a + w * part[warp + k][D + 1];
#pragma unroll
          for (int e = 0; e < kCols; ++e) sum[e] = sum[e] * a + w * part[warp + k][lane * kCols + e];
        }
      }
    }
    if (r < pairs && way == 0) {
      const size_t at = row_of(p, s, hk, pair0 + r);
      const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
      uint32_t* out = reinterpret_cast<uint32_t*>(p.o + at * D) + lane * (kCols / 2);
#pragma unroll
      for (int e = 0; e < kCols / 2; ++e) out[e] = pack_bf16(sum[2 * e] * inv, sum[2 * e + 1] * inv);
      if (lane == 0) store_lse(p, at, mm, ll);
    }
  }
}

template <int D, int NT>
cudaError_t launch_t(const CacheAttnParams& p, cudaStream_t stream) {
  constexpr int bytes = RowsLayout<D, NT>::kBytes;
  auto kernel = p.q_times != nullptr ? rows_kernel<D, NT, true> : rows_kernel<D, NT, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  kernel<<<kGrid, kThreads, bytes, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_after(join_kernel<D, NT>, dim3(kGrid - 1), 32 * kJoinWarps, 0, stream, p);
}

int tiles_of(long long rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

}  // namespace

size_t cache_rows_partial_bytes(int d, long long rows) {
  return (size_t)2 * kGrid * 8 * tiles_of(rows) * (d + 2) * sizeof(float);
}

cudaError_t launch_cache_rows(const CacheAttnParams& p, long long rows, cudaStream_t stream) {
  switch (tiles_of(rows)) {
    case 1: return p.c.d == 64 ? launch_t<64, 1>(p, stream) : launch_t<128, 1>(p, stream);
    case 2: return p.c.d == 64 ? launch_t<64, 2>(p, stream) : launch_t<128, 2>(p, stream);
    default: return p.c.d == 64 ? launch_t<64, 4>(p, stream) : launch_t<128, 4>(p, stream);
  }
}

}  // namespace h3
