// Attention over the paged int8 cache for few query rows per sequence (one
// token, a handful of drafts): per query row i of sequence b and head h, over
// the cached rows j < length[b] (causal: j <= length[b] - rows + i)
//   s_j = (q . code_j) s_k / sqrt(d) - penalty(|t_q - t_j|),
//   O = sum_j exp(s_j) code_j s_v / sum_j exp(s_j),   LSE = log sum_j exp(s_j);
// a row that sees no key gets O = 0 and LSE = -inf.
//
// A code is read once (twice for 17 to 32 pairs, then from L2) and used for the few
// rows of one sequence and K/V head: HBM-bound up to 8 pairs, from 16 on by the
// instructions per code (the same 134 MB with 8 / 16 / 32 pairs: 37 / 49 / 69 us).
// The query heads of a K/V head and the rows of a sequence form one list of
// (row, head) pairs, cut into tiles of 8 NT pairs; an item is one tile of one
// sequence and K/V head, its units are the sequence's pages.  The units of all items
// form one line that the blocks share evenly, whatever the lengths are (they are read
// on the device); a block walks its stretch item by item, and items that lie in several
// blocks are joined by a second launch from partial results (maximum, sum, unnormalised
// O in fp32).
//
// Inside a block each warp streams granules of 32 keys on its own: cp.async into
// a ring of its own (no barrier between warps until the item ends), then
//   S^T = K Q^T   mma m16n8k16 fp16, A = the codes widened exactly to fp16,
//   P^T           exp2 of the scaled scores, packed to fp16, transposed by movmatrix,
//   O^T += V^T P^T  A = the V codes, two keys of a column per register.
// fp16 and not bf16 operands, for a code widens to fp16 in two operations for
// two codes instead of three and the kernel is near the instruction rate: Q is
// scaled per row by a power of two to a maximum in [2^9, 2^10) (its 8-bit
// mantissas stay exact down to 2^-23 of the row's maximum), and the V scale goes
// into the exponent, so that a probability times its V scale is 2^12 at the row's
// largest and keeps more bits than bf16 would down to 2^-26 of that.  A V scale
// outside [2^-60, 2^40] (a page of zeros, or one marked as not finite) goes in as
// the nearest end of that range, and the product with V takes bf16 operands, whose
// range holds the rest of the scale.
// The d order of A and of Q agree by construction and nothing else sees it, so
// a lane takes 16 consecutive bytes of a row per load.  mma.sync and not tcgen05:
// 8 rows fill no 128-row tile, and the widened codes are in registers anyway.
//
// Measured, from GPU to GPU: one row of 56 heads over 116,883 rows of 8 K/V heads of 128
// (240 MB) 52 to 54 us, 32 sequences of 410 to 8,192 rows (282 MB) 59 to 64 us: 4.4 to
// 4.8 TB/s, and 4.9 to 5.4 TB/s but for the 7 us that two launches and finding the pages
// take; the same loop without its arithmetic takes 51.5 us and 60 us.  (A plain sum over
// 240 MB reads 5.3 TB/s.)  In 16-key granules, 8 warps a block: 56 and 73 us.
#include <cuda_bf16.h>

#include <type_traits>

#include "cache_attn.cuh"

namespace h3 {
namespace {

using namespace sm;

constexpr int kWarps = 6, kThreads = 32 * kWarps;
constexpr int kKeys = 32;    // keys of a granule
constexpr int kM = kKeys / 16;
constexpr int kStages = 2;
constexpr int kJoinWarps = 16;
constexpr float kRaise = 3.0f;   // log2 units: a score this far above the running maximum raises it
constexpr float kShift = 12.0f;  // a probability is 2^kShift at the running maximum: at most 2^15 in fp16
constexpr int kBlocksPerSm = 2;
constexpr int kGrid = 148 * kBlocksPerSm;
// What beginning and ending an item costs a block, in pages: it counts in the
// line, so that a block that gets many short sequences gets fewer pages (the 32
// ragged sequences: 73 us without, 68 with 1, 60 with 3, 61 with 8).
constexpr int kItemCost = 3;
constexpr int kMinShare = kItemCost + 1;

template <int D, int NT>
struct RowsLayout {
  static constexpr int kRows = 8 * NT;
  static constexpr int kV = kKeys * D;              // V codes after the K codes
  static constexpr int kMeta = 2 * kKeys * D;       // k scale, v scale, valid keys, -, then the keys' times
  static constexpr int kStage = kMeta + 16 + kKeys * 4;
  static constexpr int kPitch = D + 4;              // floats of one row of the warps' results
  static constexpr int kResult = kRows * kPitch * 4;
  // a warp's results lie over its ring
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
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
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

// Sequence b's share of the line: tiles x K/V heads x (kItemCost + pages), with
// one page at least, so that a sequence without cached rows still gets its rows
// written.
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
  s.units = s.tiles * p.c.H * (s.pages + kItemCost);
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
  Seq seq;                    // that sequence
  __device__ __forceinline__ explicit Line(const CacheAttnParams& p) {
    __shared__ long long sums[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    mine = 0;
    for (int b = tid; b < p.b.B; b += NT) {
      seq = load_seq<R>(p, b);
      mine += seq.units;
    }
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
  // The sequence that unit u lies in, its number, and the line before it.
  __device__ __forceinline__ int find(const CacheAttnParams& p, long long u, long long* before, Seq* s) const {
    __shared__ long long sums[NT / 32], at;
    __shared__ int found;
    __shared__ Seq found_seq;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (p.b.B <= NT) {
      if (u >= lo && u < lo + mine) {
        found = tid;
        found_seq = seq;
        at = lo;
      }
    } else {
      long long base = 0;
      for (int b0 = 0; b0 < p.b.B && base <= u; b0 += NT) {
        Seq mine_now{};
        if (b0 + tid < p.b.B) mine_now = load_seq<R>(p, b0 + tid);
        const long long units = mine_now.units;
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
          found_seq = mine_now;
          at = from;
        }
      }
    }
    __syncthreads();
    *before = at;
    *s = found_seq;
    return found;
  }
};

__device__ __forceinline__ long long share_of(long long total) {
  const long long even = (total + kGrid - 1) / kGrid;
  return even > kMinShare ? even : kMinShare;
}

// A block's piece of an item: pages [page0, page1) of one tile of one sequence
// and K/V head.  The first kItemCost + 1 units of an item stand for its first
// page; a piece that begins inside them has no page if there is only that one.
struct Piece1 {
  int b, hk, page0, page1, pairs;
  int i0, g0;              // query row and head of the group of the tile's first pair
  long long pair0, start;  // the tile's first pair; the line before the item
  long long end;           // the line up to the piece's end
  long long before;        // the line before the sequence
  Seq s;
  __device__ __forceinline__ int units() const { return s.pages + kItemCost; }
  __device__ __forceinline__ void cut(long long u, long long u1) {
    const int x0 = (int)(u - start), x1 = (int)min((long long)units(), u1 - start);
    page0 = x0 == 0 ? 0 : max(1, x0 - kItemCost);
    page1 = x1 == units() ? s.pages : max(1, x1 - kItemCost);
    end = start + x1;
  }
};
// The piece that unit u of the line begins, inside sequence s (`before` it).
template <int R>
__device__ __forceinline__ Piece1 piece_at(const CacheAttnParams& p, int b, const Seq& s, long long before, long long u,
                                           long long u1) {
  Piece1 w;
  w.b = b;
  w.s = s;
  w.before = before;
  const long long d = u - before;
  const int units = w.units();
  const long long item = d < 0x7FFFFFFF ? (long long)((unsigned)d / (unsigned)units) : d / units;
  const long long tile = item < 0x7FFFFFFF ? (long long)((unsigned)item / (unsigned)p.c.H) : item / p.c.H;
  w.hk = (int)(item - tile * p.c.H);
  w.start = before + item * units;
  w.cut(u, u1);
  w.pair0 = tile * R;
  w.i0 = w.g0 = 0;
  if (tile > 0) {
    w.i0 = (int)(w.pair0 / p.group);
    w.g0 = (int)(w.pair0 - (long long)w.i0 * p.group);
  }
  w.pairs = (int)min((long long)R, (long long)s.n * p.group - w.pair0);
  return w;
}
// The piece after w, which ends its item; u: its first unit.
template <int R>
__device__ __forceinline__ Piece1 piece_after(const CacheAttnParams& p, const Piece1& w, long long u, long long u1) {
  if (u < w.before + w.s.units && w.hk + 1 < p.c.H) {  // the next K/V head of the same tile
    Piece1 v = w;
    ++v.hk;
    v.start = u;
    v.cut(u, u1);
    return v;
  }
  int b = w.b;
  Seq s = w.s;
  long long before = w.before;
  while (u >= before + s.units) {
    before += s.units;
    s = load_seq<R>(p, ++b);
  }
  return piece_at<R>(p, b, s, before, u, u1);
}
// Output row (head T + packed row) of pair r of the tile.
__device__ __forceinline__ size_t row_of(const CacheAttnParams& p, const Piece1& w, int r) {
  const unsigned q = (unsigned)(w.g0 + r), i = q / (unsigned)p.group, g = q - i * (unsigned)p.group;
  return (size_t)(w.hk * p.group + (int)g) * p.b.T + w.s.first + w.i0 + (int)i;
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
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) rows_kernel(const CacheAttnParams p) {
  using L = RowsLayout<D, NT>;
  constexpr int R = L::kRows, kJ = D / 16;
  constexpr bool kQRegs = NT == 1;  // Q fragments in registers, else read from shared memory
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * L::kRing;
  const uint32_t ring_a = smem_u32(ring), q_a = smem_u32(smem + L::kQ);
  float2* ml = reinterpret_cast<float2*>(smem + L::kMl);  // [warp][R] (maximum, sum)

  wait_dependency();
  launch_dependents();
  const Line<R, kThreads> line(p);
  const long long total = line.total, share = share_of(total);
  const long long u0 = blockIdx.x * share, u1 = min(total, u0 + share);
  if (u0 >= u1) return;
  long long before;
  Seq s0;
  const int b0 = line.find(p, u0, &before, &s0);
  Piece1 w = piece_at<R>(p, b0, s0, before, u0, u1);
  if (w.page0 >= w.page1) {  // the rest of an item of one page, which the block before has
    if (w.end >= u1) return;
    w = piece_after<R>(p, w, w.end, u1);
  }

  // this warp's granules of the piece: keys first, first + kWarps * kKeys, ... < end
  int end, first, steps;
  auto begin = [&]() {
    end = min(w.s.len, w.page1 * kBlock);
    first = w.page0 * kBlock + warp * kKeys;
    steps = first < end ? (end - first + kWarps * kKeys - 1) / (kWarps * kKeys) : 0;
  };
  auto issue = [&](int i) {
    if (i < steps) {
      const int key = first + i * (kWarps * kKeys);
      const int page = page_id(p.c, p.b, w.b, key / kBlock, p.status);
      const uint32_t st = ring_a + i % kStages * L::kStage;
      if (page >= 0) {
        const size_t at = (size_t)page * p.c.H + w.hk;
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
  // Q of the piece's tile (8 columns n = pairs; k = the columns of a word of codes)
  uint4 qw[D / 32];
  auto load_q = [&]() {
    const int r = (kQRegs ? 0 : warp * 8) + g;
    const uint16_t* src = nullptr;
    if ((kQRegs || warp < NT) && r < w.pairs) {
      const unsigned q = (unsigned)(w.g0 + r), i = q / (unsigned)p.group, gg = q - i * (unsigned)p.group;
      src = p.q + (w.hk * p.group + (int)gg) * p.q_head + (long long)(w.s.first + w.i0 + (int)i) * p.q_row + t * 16;
    }
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
      qw[c] = src != nullptr ? __ldg(reinterpret_cast<const uint4*>(src + c / 2 * 64) + (c & 1)) : make_uint4(0u, 0u, 0u, 0u);
  };
  begin();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);
  load_q();

  while (true) {
    uint32_t qf[kQRegs ? 2 * kJ : 1];
    if (kQRegs || warp < NT) {
      const int r = (kQRegs ? 0 : warp * 8) + g;
      float y[D / 4], top = 0.0f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const uint32_t x[4] = {qw[c].x, qw[c].y, qw[c].z, qw[c].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[8 * c + 2 * i] = __uint_as_float(x[i] << 16);
          y[8 * c + 2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
          top = fmaxf(top, fmaxf(fabsf(y[8 * c + 2 * i]), fabsf(y[8 * c + 2 * i + 1])));
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
    int lim[NT][2], lim_all = w.s.len;
    float tq[NT][2], qs[NT][2];
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * x + 2 * t + e;
        lim[x][e] = w.s.len;
        tq[x][e] = NAN;
        qs[x][e] = reinterpret_cast<const float*>(smem + L::kQScale)[r] * p.scale_log2;
        if (r < w.pairs) {
          const int i = w.i0 + (int)((unsigned)(w.g0 + r) / (unsigned)p.group);
          if (p.causal) lim[x][e] = min(w.s.len, max(0, w.s.len - w.s.n + i + 1));
          if (kPen) tq[x][e] = __ldg(p.q_times + w.s.first + i);
        }
        lim_all = min(lim_all, lim[x][e]);
      }
    lim_all = __reduce_min_sync(kFull, lim_all);

    float o[NT][kJ][4] = {}, m[NT][2], l[NT][2] = {};
#pragma unroll
    for (int x = 0; x < NT; ++x) m[x][0] = m[x][1] = -INFINITY;

    for (int i = 0; i < steps; ++i) {
      cp_async_wait<kStages - 2>();
      __syncwarp();  // every lane's copies of this stage have landed, and the stage issued next is read
      issue(i + kStages - 1);
      const uint32_t st = ring_a + i % kStages * L::kStage;
      const float* meta = reinterpret_cast<const float*>(ring + i % kStages * L::kStage + L::kMeta);
      const int live = __float_as_int(meta[2]);
      if (live == 0) continue;
      // the V scale's part in the exponent (the lower end for NaN), and what of it stays outside
      const float ks = meta[0], vs = meta[1], ve = fminf(fmaxf(vs, kScaleLow), kScaleHigh);
      const float lv = log2_approx(ve), iv = rcp_approx(ve);
      const int key = first + i * (kWarps * kKeys);

      // S^T: kKeys keys x 8 NT pairs
      float acc[kM][NT][4] = {};
#pragma unroll
      for (int mt = 0; mt < kM; ++mt)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const uint32_t a = st + (16 * mt + g) * D + (D == 128 ? (4 * c + t) ^ ((g & 1) << 2) : t) * 16;
          const uint4 wa = lds128(a), wb = lds128(a + 8 * D);
          const uint32_t ra[4] = {wa.x, wa.y, wa.z, wa.w}, rb[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            const uint32_t a0 = widen2h(ra[i4]), a1 = widen2h(rb[i4]);
            const uint32_t a2 = widen2h(ra[i4] >> 8), a3 = widen2h(rb[i4] >> 8);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              uint2 f;
              if constexpr (kQRegs) f = make_uint2(qf[2 * (4 * c + i4)], qf[2 * (4 * c + i4) + 1]);
              else f = lds64(q_a + (((4 * c + i4) * NT + x) * 32 + lane) * 8);
              mma_f16(acc[mt][x], a0, a1, a2, a3, f.x, f.y);
            }
          }
        }
      // scores times V scales in log2 units: [x][0], [x][1] key g, [x][2], [x][3] key g + 8 of a 16
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        const float c0 = qs[x][0] * ks, c1 = qs[x][1] * ks;
#pragma unroll
        for (int mt = 0; mt < kM; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = fmaf(acc[mt][x][e], e & 1 ? c1 : c0, lv);
            if (kPen) {
              const float dt = fabsf(tq[x][e & 1] - meta[4 + 16 * mt + g + (e >> 1) * 8]);
              const float ex = fmaxf(dt - p.window, 0.0f) * p.inv_falloff;
              v -= fminf(p.strength_log2 * ex * ex, p.cap_log2);
            }
            acc[mt][x][e] = v;
          }
      }
      if (key + live > lim_all || live < kKeys) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int mt = 0; mt < kM; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int kk = 16 * mt + g + (e >> 1) * 8;
              if (kk >= live || key + kk >= lim[x][e & 1]) acc[mt][x][e] = -INFINITY;
            }
      }
      // a score kRaise above its pair's running maximum raises it
      bool over = false;
      float top[NT][2];
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(acc[0][x][e], acc[0][x][e + 2]);
#pragma unroll
          for (int mt = 1; mt < kM; ++mt) mx = max3f(mx, acc[mt][x][e], acc[mt][x][e + 2]);
          top[x][e] = mx;
          over = over || mx > m[x][e] + kRaise;
        }
      if (__any_sync(kFull, over)) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = top[x][e];
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
      // probabilities, and O^T += V^T P^T; `outside`: the scale has a rest
      auto accumulate = [&](auto outside, float rest) {
        constexpr bool kOutside = decltype(outside)::value;
        // a rest that is not finite stays away from pairs that do not see the key
        auto packed = [&](float a, float b) {
          if constexpr (kOutside) return pack_bf16(a == 0.0f ? 0.0f : a * rest, b == 0.0f ? 0.0f : b * rest);
          else return pack_f16(a, b);
        };
        auto widened = [&](uint32_t w) {
          if constexpr (kOutside) return widen2(w);
          else return widen2h(w);
        };
        uint32_t pb[kM][NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          const float m0 = (m[x][0] == -INFINITY ? 0.0f : m[x][0]) - kShift;
          const float m1 = (m[x][1] == -INFINITY ? 0.0f : m[x][1]) - kShift;
          float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
          for (int mt = 0; mt < kM; ++mt) {
            const float p0 = ex2(acc[mt][x][0] - m0), p1 = ex2(acc[mt][x][1] - m1);
            const float p2 = ex2(acc[mt][x][2] - m0), p3 = ex2(acc[mt][x][3] - m1);
            s0 += p0 + p2;
            s1 += p1 + p3;
            pb[mt][x][0] = transpose8x8(packed(p0, p1));
            pb[mt][x][1] = transpose8x8(packed(p2, p3));
          }
          l[x][0] = fmaf(s0, iv, l[x][0]);
          l[x][1] = fmaf(s1, iv, l[x][1]);
        }
        // this lane's keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of a 16, its columns from g D / 8 on
#pragma unroll
        for (int mt = 0; mt < kM; ++mt) {
          uint32_t v[4][D / 32];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 2 * t + (r & 1) + (r >> 1) * 8;
            const uint32_t a = st + L::kV + (16 * mt + row) * D;
            if constexpr (D == 128) {
              const uint4 x = lds128(a + ((g ^ ((row >> 1 & 3) << 1)) << 4));
              v[r][0] = x.x, v[r][1] = x.y, v[r][2] = x.z, v[r][3] = x.w;
            } else {
              const uint2 x = lds64(a + (((g >> 1) ^ (row >> 1 & 3)) << 4) + (g & 1) * 8);
              v[r][0] = x.x, v[r][1] = x.y;
            }
          }
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            const uint32_t sel = j & 1 ? 0x7632 : 0x5410;
            const uint32_t ab = __byte_perm(v[0][j >> 1], v[1][j >> 1], sel);
            const uint32_t cd = __byte_perm(v[2][j >> 1], v[3][j >> 1], sel);
            const uint32_t a0 = widened(ab), a1 = widened(ab >> 8), a2 = widened(cd), a3 = widened(cd >> 8);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              if constexpr (kOutside) mma_bf16(o[x][j], a0, a1, a2, a3, pb[mt][x][0], pb[mt][x][1]);
              else mma_f16(o[x][j], a0, a1, a2, a3, pb[mt][x][0], pb[mt][x][1]);
            }
          }
        }
      };
      if (ve == vs) accumulate(std::false_type{}, 1.0f);
      else accumulate(std::true_type{}, vs * iv);
    }
    __syncwarp();  // the ring is read

    // on to the next piece: its Q loads while this one is joined
    const Piece1 done = w;
    const long long u = w.end;
    const bool more = u < u1;
    if (more) {
      w = piece_after<R>(p, w, u, u1);
      begin();
    }
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
    if (more) load_q();
    __syncthreads();
    const bool whole = done.page0 == 0 && done.page1 == done.s.pages;
    float* slot = whole ? nullptr : slot_of<D, R>(p, blockIdx.x, done.page0 > 0 ? 0 : 1);
    for (int i = tid; i < R * (D / 4); i += kThreads) {
      const int r = i / (D / 4), col = i % (D / 4) * 4;
      if (r >= done.pairs) break;
      float mm = -INFINITY, ll = 0.0f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) mm = fmaxf(mm, ml[x * R + r].x);
      float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float2 v = ml[x * R + r];
        const float a = v.x == -INFINITY ? 0.0f : ex2(v.x - mm);
        const float4 y = *reinterpret_cast<const float4*>(smem + x * L::kRing + (r * L::kPitch + col) * 4);
        ll += a * v.y;
        sum.x += a * y.x, sum.y += a * y.y, sum.z += a * y.z, sum.w += a * y.w;
      }
      if (whole) {
        const size_t at = row_of(p, done, r);
        store_cols(p, at, col, sum, ll == 0.0f ? 0.0f : 1.0f / ll);
        if (col == 0) store_lse(p, at, mm, ll);
      } else {
        *reinterpret_cast<float4*>(slot + r * D + col) = sum;
        if (col == 0) *reinterpret_cast<float2*>(slot + R * D + 2 * r) = make_float2(mm, ll);
      }
    }
    if (!more) break;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);
  }
  cp_async_wait<0>();
}

// Joins the items that several blocks share: block x stands for the border
// between the stretches x and x + 1 and works on the item that lies across it;
// the blocks of an item's borders take its pairs in turn, and a block's warps
// share a pair's slots.  A lane holds D / 32 columns.
template <int D, int NT>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const CacheAttnParams p) {
  constexpr int R = 8 * NT, kCols = D / 32;
  using Cols = typename std::conditional<kCols == 4, float4, float2>::type;
  __shared__ float part[kJoinWarps][D + 2];
  const Line<R, 32 * kJoinWarps> line(p);
  const long long total = line.total, share = share_of(total);
  const long long u = (blockIdx.x + 1) * share;
  if (u >= total) {
    wait_dependency();
    return;
  }
  long long before;
  Seq s;
  const int b = line.find(p, u, &before, &s);
  const Piece1 w = piece_at<R>(p, b, s, before, u, total);
  wait_dependency();
  if (w.start == u || w.s.pages == 1) return;  // the border lies between two items, or one block has all of it
  const long long c0 = w.start / share;
  const int n = (int)((w.start + w.units() - 1) / share - c0) + 1;    // slots: n - 1 borders
  const int turn = (int)(blockIdx.x - c0);
  const int rows = turn < w.pairs ? (w.pairs - turn + n - 2) / (n - 1) : 0;  // pairs turn, turn + n - 1, ...
  const int ways = rows > 0 ? max(1, kJoinWarps / rows) : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, way = warp % ways;
  auto slot = [&](int c) { return slot_of<D, R>(p, c0 + c, c == 0 ? 1 : 0); };
  for (int k0 = 0; k0 < rows; k0 += kJoinWarps / ways) {
    const int k = k0 + warp / ways, r = turn + k * (n - 1);
    const bool mine = k < rows && warp / ways < kJoinWarps / ways;
    float mm = -INFINITY, ll = 0.0f, sum[kCols] = {};
    if (mine)
      for (int c = way; c < n; c += 32 * ways) {  // 32 slots at a time, a lane for each
        const int at = c + lane * ways;
        const float2 x = at < n ? *reinterpret_cast<const float2*>(slot(at) + R * D + 2 * r)
                                : make_float2(-INFINITY, 0.0f);
        float mn = fmaxf(mm, x.x);
#pragma unroll
        for (int q = 16; q > 0; q >>= 1) mn = fmaxf(mn, __shfl_xor_sync(kFull, mn, q));
        const float base = mn == -INFINITY ? 0.0f : mn, a = ex2(mm - base), e_c = ex2(x.x - base);
        float lw = e_c * x.y;
#pragma unroll
        for (int q = 16; q > 0; q >>= 1) lw += __shfl_xor_sync(kFull, lw, q);
        mm = mn;
        ll = ll * a + lw;
#pragma unroll
        for (int e = 0; e < kCols; ++e) sum[e] *= a;
        const int live = min(32, (n - c + ways - 1) / ways);
#pragma unroll 8
        for (int q = 0; q < live; ++q) {
          const float wq = __shfl_sync(kFull, e_c, q);
          const Cols y = *(reinterpret_cast<const Cols*>(slot(c + q * ways) + r * D) + lane);
          const float* yy = reinterpret_cast<const float*>(&y);
#pragma unroll
          for (int e = 0; e < kCols; ++e) sum[e] = fmaf(wq, yy[e], sum[e]);
        }
      }
    if (ways > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kCols; ++e) part[warp][lane * kCols + e] = sum[e];
      if (lane == 0) part[warp][D] = mm, part[warp][D + 1] = ll;
      __syncthreads();
      if (mine && way == 0)
        for (int q = 1; q < ways; ++q) {
          const float mk = part[warp + q][D], mn = fmaxf(mm, mk), base = mn == -INFINITY ? 0.0f : mn;
          const float a = ex2(mm - base), e_q = ex2(mk - base);
          mm = mn;
          ll = ll * a + e_q * part[warp + q][D + 1];
#pragma unroll
          for (int e = 0; e < kCols; ++e) sum[e] = sum[e] * a + e_q * part[warp + q][lane * kCols + e];
        }
    }
    if (mine && way == 0) {
      const size_t at = row_of(p, w, r);
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
  if ((e = launch_after(kernel, dim3(kGrid), kThreads, bytes, stream, p)) != cudaSuccess) return e;
  return launch_after(join_kernel<D, NT>, dim3(kGrid - 1), 32 * kJoinWarps, 0, stream, p);
}

// Tiles of 8 pairs where no sequence has more, else of 16.  Two sequences of 16,384
// rows, 16 heads of 128, with tiles of 8 / 16 / 32 pairs: 8 pairs take 33 / 47 / 69 us,
// 16 pairs 51 / 49 / 70 us, 32 pairs 88 / 68 / 72 us (a tile of 32 leaves one block
// on an SM; two of 16 read the codes again, from L2).
int tiles_of(long long pairs) { return pairs <= 8 ? 1 : 2; }

}  // namespace

size_t cache_rows_partial_bytes(int d, long long pairs) {
  return (size_t)2 * kGrid * 8 * tiles_of(pairs) * (d + 2) * sizeof(float);
}

cudaError_t launch_cache_rows(const CacheAttnParams& p, long long pairs, cudaStream_t stream) {
  if (tiles_of(pairs) == 1) return p.c.d == 64 ? launch_t<64, 1>(p, stream) : launch_t<128, 1>(p, stream);
  return p.c.d == 64 ? launch_t<64, 2>(p, stream) : launch_t<128, 2>(p, stream);
}

}  // namespace h3
