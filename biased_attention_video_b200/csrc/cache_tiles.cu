// Attention over the paged int8 cache for many query rows per sequence, on the
// tensor cores (tcgen05); the formulas are those of cache_rows.cu.
//
// The (query row, head of the group) pairs of a sequence and K/V head form one
// list, row by row, cut into tiles of 256 pairs: two tcgen05 tiles A and B of
// 128 rows that share every K and V block, so that a code is widened to bf16
// once for 256 rows.  A step takes 128 keys (two pages): a product S = Q K^T of
// N = 128 keys runs in 64 cycles, one of N = 64 in 48.  While the softmax works on
// one tile's scores the tensor cores run the other's products.
//
// Warp roles (512 threads, one block per SM; the 128 registers a thread that the
// block starts with are dealt out anew, 160 / 112 / 80 per warpgroup):
//   warps 0..3, 4..7  softmax of tile A, B: one thread per pair (= TMEM lane);
//                     they also bring Q in and the output out
//   warps 8..11       keys and values: 16-byte loads of codes, held one step ahead
//                     in registers, widened and stored as bf16 in the swizzled
//                     layout the products read (two buffers of K and of V)
//   warp 12           TMEM owner and tcgen05.mma issuer; warp 13 finds the items
//                     (14, 15 idle)
//
// TMEM (512 columns): S_A [0, 128), S_B [128, 256), O_A from 256, O_B from 256 + d.
// The bf16 probabilities go over the first 64 columns of their S.  Issue order:
//   S_A(0) S_B(0) | PV_A(0) S_A(1) | PV_B(0) S_B(1) | PV_A(1) S_A(2) | ...
// The products of one thread run in order: S_A(j+1) does not overwrite P_A(j)
// before PV_A(j) has read it, and when S_A(j+1) is complete so is PV_A(j), so a
// rescale of O_A needs no wait of its own.
//
// The issuer is on the critical path and every barrier it touches costs it 150 to
// 200 cycles (a commit right behind another one 500 to 1000), so it waits three
// times a step (the next keys, the probabilities of A and of B) and commits twice
// (the scores of A and of B); all else follows from the order: the scores of step j
// being complete, its keys and the values of step j - 1 are free again.
//
// The columns of K, V and Q are stored with every group of four in the order
// (0, 2, 1, 3), as the codes widen; the products do not see it, and O comes back
// in the same order.
//
// Work split: an item is one tile of one sequence and K/V head, its steps go up to
// the last key that any of its rows sees.  All items form one line, sequence by
// sequence, head by head, tile by tile; the blocks share it evenly, and an item
// that lies in several blocks is joined by another launch from partial results
// (maximum, sum, unnormalised O in fp32).  The line is laid out on the device
// (plan_kernel), for the lengths are read there.
//
// Measured, from GPU to GPU: 2,126 rows of 8 heads of 128 over 57,402 rows with the penalty
// 617 to 645 us (775 to 810 TFLOP/s), causal chunks of four sequences of up to 2,500
// rows, 16 heads on 4, 334 to 352 us (695 to 735), 70 rows of 16 heads over 16,384 rows
// of two sequences 82 us.  What bounds it is latency: a step takes about 4,400 cycles,
// its products 2,050; a tile's scores, softmax (about 2,500 with both tiles at it) and
// products follow one another, and the two tiles cover each other only in part.
#include <cuda_bf16.h>

#include <type_traits>

#include "cache_attn.cuh"

namespace h3 {
namespace {

using namespace sm;

constexpr int kThreads = 512;
constexpr int kMmaWarp = 12;
constexpr int kWidenWarp = 8;
constexpr int kTile = 256;   // pairs of an item
constexpr int kStep = 128;   // keys of a step
constexpr int kGrid = 148;   // one block per SM
// What beginning and ending an item costs (Q, the wait for the first step, the
// output), in steps: it counts in the line.  With 0 / 2 / 4 / 6 / 8 / 12 the causal
// chunks take 374 / 350 / 343 / 337 / 331 / 337 us, 120 rows of 16 sequences of up to
// 1,200 50 / 47 / 46 / 44 / 44 / 44 us, 70 rows over 16,384 86 / 84 / 82 / 82 / 85 / 86 us.
constexpr int kItemCost = 6;
constexpr long long kMinShare = kItemCost + 2;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 256;

// ---------------------------------------------------------------- the line

struct Seq {
  int first, n, len, tiles;
};
__device__ __forceinline__ Seq load_seq(const CacheAttnParams& p, int b) {
  Seq s;
  const SeqRows r = seq_rows(p.b, b, p.status);
  s.first = r.first;
  s.n = r.n;
  s.len = seq_length(p.b, b, p.status);
  s.tiles = (int)(((long long)s.n * p.group + kTile - 1) / kTile);
  return s;
}
// Steps of tile t (one at least, so that rows that see nothing are written too).
__device__ __forceinline__ int tile_steps(const CacheAttnParams& p, const Seq& s, int t) {
  int seen = s.len;
  if (p.causal) {
    const long long pairs = (long long)s.n * p.group, last = min(pairs, (long long)(t + 1) * kTile) - 1;
    seen = max(0, min(s.len, s.len - s.n + (int)(last / p.group) + 1));
  }
  return max(1, (seen + kStep - 1) / kStep);
}

// The step that unit x of an item begins (0 <= x <= kItemCost + steps).
__device__ __forceinline__ int step_at(int x, int steps) { return min(steps, max(0, x - kItemCost)); }

// base[b]: the line before sequence b; base[B]: its length.  One block, one warp
// per sequence at a time.
__global__ void __launch_bounds__(1024) plan_kernel(const CacheAttnParams p) {
  __shared__ long long units[32];
  __shared__ long long before;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  launch_dependents();
  if (threadIdx.x == 0) {
    before = 0;
    p.base[0] = 0;
  }
  for (int b0 = 0; b0 < p.b.B; b0 += 32) {
    const int b = b0 + warp;
    long long u = 0;
    if (b < p.b.B) {
      const Seq s = load_seq(p, b);
      if (p.causal) {
        for (int t = lane; t < s.tiles; t += 32) u += kItemCost + tile_steps(p, s, t);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(kFull, u, o);
      } else {
        u = (long long)s.tiles * (kItemCost + tile_steps(p, s, 0));
      }
    }
    if (lane == 0) units[warp] = u * p.c.H;
    __syncthreads();
    if (warp == 0) {
      long long v = units[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long w = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += w;
      }
      const long long at = before + v;
      if (b0 + lane < p.b.B) p.base[b0 + lane + 1] = at;
      __syncwarp();
      if (lane == 31) before = at;
    }
    __syncthreads();
  }
}

// The item that unit u lies in, found by one warp; every lane gets it.
struct Item {
  int b, hk, first, n, len;
  long long pair0;
  int pairs;         // of the tile
  int steps;         // of the whole item
  long long start;   // the line before the item
  __device__ __forceinline__ int units() const { return kItemCost + steps; }
  __device__ __forceinline__ int step(long long u) const {
    return step_at((int)max(0ll, min((long long)units(), u - start)), steps);
  }
};
__device__ __forceinline__ Item find_item(const CacheAttnParams& p, long long u) {
  const int lane = threadIdx.x & 31;
  Item it;
  int b = 0;  // the last sequence whose line begins at or before u; base ascends
  for (int span = p.b.B; span > 1;) {
    const int step = (span + 31) / 32, at = b + lane * step;
    const unsigned in = __ballot_sync(kFull, lane * step < span && p.base[at] <= u);
    const int last = in != 0u ? 31 - __clz(in) : 0;
    b += last * step;
    span = min(step, span - last * step);
  }
  const Seq s = load_seq(p, b);
  const long long lo = p.base[b], per_head = (p.base[b + 1] - lo) / p.c.H;
  it.b = b;
  it.first = s.first;
  it.n = s.n;
  it.len = s.len;
  it.hk = (int)((u - lo) / per_head);
  const long long head_lo = lo + it.hk * per_head;
  int t = 0;
  if (!p.causal) {
    it.steps = tile_steps(p, s, 0);
    t = (int)((u - head_lo) / it.units());
    it.start = head_lo + (long long)t * it.units();
  } else {
    long long at = head_lo;
    it.start = head_lo;
    for (int t0 = 0; t0 < s.tiles; t0 += 32) {
      const int mine = t0 + lane < s.tiles ? kItemCost + tile_steps(p, s, t0 + lane) : 0;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned past = __ballot_sync(kFull, mine > 0 && u < at + incl);
      if (past != 0u) {
        const int l = __ffs(past) - 1;
        t = t0 + l;
        it.start = at + __shfl_sync(kFull, incl - mine, l);
        break;
      }
      at += __shfl_sync(kFull, incl, 31);
    }
    it.steps = tile_steps(p, s, t);
  }
  it.pair0 = (long long)t * kTile;
  it.pairs = (int)min((long long)kTile, (long long)s.n * p.group - it.pair0);
  return it;
}

__device__ __forceinline__ long long share_of(long long total) {
  const long long even = (total + kGrid - 1) / kGrid;
  return even > kMinShare ? even : kMinShare;
}

// Slot of partial results: unnormalised O [256][D], then (maximum, sum) [256].
// Block c's slot 0 holds an item that an earlier block began, slot 1 the item
// that it begins and a later one goes on with.
template <int D>
__device__ __forceinline__ float* slot_of(const CacheAttnParams& p, long long block, int which) {
  return p.partial + (2 * block + which) * (size_t)(kTile * (D + 2));
}

// --------------------------------------------------------------- the kernel

// What the softmax needs to know of a page.
struct PageMeta {
  float c;      // K scale, log2 units: score = c * (q . code)
  float lv;     // log2 of the V scale
  float iv, vs; // 1 / V scale, V scale
  int live;     // valid keys: 0 for a page past the end or outside the cache
  int mode;     // guide times of its keys: 0 none, 1 all the same (t), 2 several
  float t;
  int plain;    // 64 valid keys, V scale in the range in which it goes into the exponent
};
// A score may exceed the running maximum by this much (log2 units) before the
// maximum is brought up: probabilities, sums and O are floating point, so a stale
// maximum costs no accuracy, and one pass over the scores is enough.  (Probabilities
// are rounded to bf16 for the product, 2^-8 of each; their sum is not.)
constexpr float kStale = 60.0f;

template <int D>
struct TilesLayout {
  static constexpr int kHalves = D / 64;       // 128-byte swizzle atoms along d
  static constexpr int kAtom = 128 * 128;      // one 128-byte-wide column of 128 rows
  static constexpr int kBlockBytes = kHalves * kAtom;  // a Q tile, a K or V block
  static constexpr int kQ = 0;                 // tiles A, B
  static constexpr int kK = 2 * kBlockBytes;   // two buffers
  static constexpr int kV = 4 * kBlockBytes;   // two buffers
  static constexpr int kMetaSlots = 4;
  static constexpr int kMeta = 6 * kBlockBytes;                // [4] x 2 pages
  static constexpr int kTimes = kMeta + kMetaSlots * 2 * (int)sizeof(PageMeta);  // [4][128]
  static constexpr int kBars = kTimes + kMetaSlots * kStep * 4;
  static constexpr int kNumBars = 2 + 1 + 4 + 1 + 4 + 2 + 1 + 1;
  static constexpr int kMisc = kBars + kNumBars * 8;  // TMEM base, abort flag
  static constexpr int kItem = kMisc + 16;
  static constexpr int kBytes = 1024 + kItem + (int)sizeof(Item) + 16;
};

// wait_bar by a whole warp, with one answer
template <bool kSuspend, class Params>
__device__ __forceinline__ bool wait_bar_all(uint64_t* bar, uint32_t parity, const Params& p, volatile int* abort) {
  return __all_sync(kFull, wait_bar<kSuspend>(bar, parity, p, abort));
}

// The whole block, from roles that run different code.
__device__ __forceinline__ void block_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

// kSuspend false: for calls with a poll limit (h3attn_set_wait_polls), whose polls must
// not suspend: one that does outlasts every wait here, so that no limit would run out.
// (One kernel that looks at the limit at every wait is 8 to 13 % slower.)
template <int D, bool kPen, bool kSuspend>
__global__ void __launch_bounds__(kThreads, 1) tiles_kernel(const CacheAttnParams p) {
  using L = TilesLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t *k_full = bar, *v_full = bar + 2, *m_full = bar + 3, *q_full = bar + 7, *s_full = bar + 8,
           *p_full = bar + 12, *o_final = bar + 14, *drain = bar + 15;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  Item* item_slot = reinterpret_cast<Item*>(smem + L::kItem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  wait_dependency();
  launch_dependents();  // after the wait: the join reads the line, too, before it waits for this kernel
  const long long total = p.base[p.b.B], share = share_of(total);
  const long long u0 = blockIdx.x * share, u1 = min(total, u0 + share);
  if (u0 >= u1) return;
  // an earlier call or block that gave up leaves the status word set
  if (tid == 0) *abort_flag = *reinterpret_cast<volatile int*>(p.status) == kStatusTimeout ? 1 : 0;
  __syncthreads();
  if (*abort_flag) return;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, 4);
      mbar_init(s_full + i, 1);
      mbar_init(s_full + 2 + i, 1);
      mbar_init(p_full + i, 4);
    }
    for (int i = 0; i < L::kMetaSlots; ++i) mbar_init(m_full + i, 4);
    mbar_init(v_full, 4);
    mbar_init(q_full, 8);
    mbar_init(o_final, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Every role walks the block's items in step.  next(): the next item, the same
  // for all (found by the first warp of the idle ones), or false at the end or
  // after a give-up.
  long long u = u0;
  Item it;
  int step0 = 0, n = 0;
  int subs = 0;  // tiles that have rows
  bool began = false;  // began: the item's first unit is this block's
  uint32_t items = 0;                        // items before
  uint32_t done = 0, done_b = 0;             // their steps, and the steps of those with a tile B
  auto next = [&]() -> bool {
    if (n > 0) {
      ++items;
      done += (uint32_t)n;
      if (subs == 2) done_b += (uint32_t)n;
    }
    // every role is done with the last item's buffers
    __syncwarp();
    tc_fence_before();
    block_sync();
    tc_fence_after();
    if (*abort_flag) return false;
    for (n = 0; n == 0; u = it.start + it.units()) {  // a stretch may touch an item without a step of it
      if (u >= u1) return false;
      if (warp == kMmaWarp + 1) {
        const Item x = find_item(p, u);
        if (lane == 0) *item_slot = x;
        __syncwarp();
      }
      block_sync();
      it = *item_slot;
      block_sync();
      step0 = it.step(u);
      n = it.step(u1) - step0;
      subs = it.pairs > 128 ? 2 : 1;
      began = u == it.start;
    }
    return true;
  };

  // 2 x 128 x 160 + 128 x 112 + 128 x 80 = 512 x 128 registers
  if (warp < kWidenWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    while (next()) {
      // --------------------------------------------- Q, softmax, output
      const int sub = warp >> 2, r = tid & 127;  // r: row of the tile = TMEM lane
      const int pr = sub * 128 + r;
      const bool valid = pr < it.pairs;
      // pair pr of the tile: its query row and head
      const int i0 = (int)(it.pair0 / p.group), g0 = (int)(it.pair0 % p.group) + (valid ? pr : 0);
      const int row = i0 + g0 / p.group, head = it.hk * p.group + g0 % p.group;
      {
        const uint16_t* src = p.q + head * p.q_head + (long long)(it.first + row) * p.q_row;
        uint8_t* dst = smem + L::kQ + sub * L::kBlockBytes + r * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (valid) w = __ldg(reinterpret_cast<const uint4*>(src) + c);
          *reinterpret_cast<uint4*>(dst + (c >> 3) * L::kAtom + (((c & 7) ^ (r & 7)) << 4)) =
              make_uint4(__byte_perm(w.x, w.y, 0x5410), __byte_perm(w.x, w.y, 0x7632),
                         __byte_perm(w.z, w.w, 0x5410), __byte_perm(w.z, w.w, 0x7632));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      if (sub < subs) {
        const int lim = valid && p.causal ? max(0, min(it.len, it.len - it.n + row + 1)) : it.len;
        const int lim_all = __reduce_min_sync(kFull, lim);
        const float tq = kPen && valid ? __ldg(p.q_times + it.first + row) : NAN;
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lane_addr + (uint32_t)(128 * sub);
        const uint32_t t_o = tmem + lane_addr + kTmemO + (uint32_t)(D * sub);
        float m = -INFINITY, l = 0.0f;
        bool ok = true, warm = false;  // warm: every row of the warp has a running maximum

        // The running maximum becomes at least mx - 8; O and l follow by the factor
        // that is returned, a power of two.  TMEM stores are asynchronous, and only
        // tmem_wait_st() orders a later load of the same columns behind them: it covers
        // the O that an earlier raise of the same step stored, which is loaded here, and
        // the probabilities that the step has stored, which the caller loads back.
        auto raise = [&](float mx) -> float {
          tmem_wait_st();
          const bool grow = mx > m + kRescaleThreshold;
          const bool rescale = grow && m > -INFINITY;
          const float up = rescale ? ceilf(mx - m) : 0.0f;
          const float alpha = ex2(-up);
          if (grow) m = rescale ? m + up : mx;
          if (__any_sync(kFull, rescale)) {
            l *= alpha;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              float x[32];
              uint32_t y[32];
              __syncwarp();
              tmem_ld32f(t_o + c * 32, x);
              tmem_landed(x);
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(x[i] * alpha);
              tmem_st32(t_o + c * 32, y);
            }
          }
          return alpha;
        };

        auto top32 = [&](const float (&s)[32]) -> float {
          float mp[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) mp[i] = fmaxf(s[i], s[i + 4]);
#pragma unroll
          for (int i = 8; i < 32; i += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) mp[e] = max3f(mp[e], s[i + e], s[i + 4 + e]);
          return fmaxf(max3f(mp[0], mp[1], mp[2]), mp[3]);
        };

        for (int j = 0; ok && j < n; ++j) {
          const uint32_t q = done + j, mine = (sub ? done_b : done) + j;  // steps, and steps of this tile
          const int slot = q & 3;
          ok = wait_bar_all<kSuspend>(m_full + slot, (q >> 2) & 1u, p, abort_flag);
          if (!ok) break;
          const PageMeta* meta = reinterpret_cast<const PageMeta*>(smem + L::kMeta) + 2 * slot;
          const PageMeta pa = meta[0], pb = meta[1];
          const float* times = reinterpret_cast<const float*>(smem + L::kTimes) + slot * kStep;
          const int key0 = (step0 + j) * kStep;
          const bool plain = pa.plain && pb.plain && key0 + kStep <= lim_all;
          const float pen_a = kPen && pa.mode == 1 ? block_penalty_log2(tq, pa.t, p) : 0.0f;
          const float pen_b = kPen && pb.mode == 1 ? block_penalty_log2(tq, pb.t, p) : 0.0f;
          ok = wait_bar_all<kSuspend>(s_full + 2 * sub + (mine & 1u), (mine >> 1) & 1u, p, abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (plain) {
            float x[32], y[32];
            uint32_t pk[32];
            auto load32 = [&](float (&to)[32], int col) {
              __syncwarp();
              tmem_ld32f(t_s + col, to);
            };
            auto probs32 = [&](const float (&s)[32], float off, float c, uint32_t* to) -> float {
              return probs16_fast(s, off, c, to) + probs16_fast(s + 16, off, c, to + 8);
            };
            // one page with the running maximum as it is; false if a score exceeds it by 2^kStale
            auto page = [&](int col, const PageMeta& pg, float pen, bool more) -> bool {
              const float off = pg.lv - (m + pen);  // m + pen first: both may be large
              tmem_landed(x);
              load32(y, col + 32);
              float top = top32(x), s = probs32(x, off, pg.c, pk);
              tmem_landed(y);
              if (more) load32(x, col + 64);
              top = fmaxf(top, top32(y));
              s += probs32(y, off, pg.c, pk + 16);
              if (__any_sync(kFull, top * pg.c - pen > m + kStale)) return false;
              l = fmaf(s, pg.iv, l);
              __syncwarp();
              tmem_st32(t_s + col / 2, pk);
              return true;
            };
            load32(x, 0);
            const bool first = warm && page(0, pa, pen_a, true);  // the first page's probabilities are stored
            warm = first && page(64, pb, pen_b, false);
            if (!warm) {
              // bring the maximum up first: over both pages, or over the second one when the first is stored
              float mx = m;
              tmem_landed(x);
              for (int c = first ? 64 : 0; c < 128; c += 32) {
                load32(x, c);
                tmem_landed(x);
                mx = fmaxf(mx, top32(x) * (c < 64 ? pa.c : pb.c) - (c < 64 ? pen_a : pen_b));
              }
              const float alpha = raise(mx);
              if (first) {
                uint32_t w[32];
                tmem_ld32(t_s, w);
                tmem_landed(w);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  w[i] = pack_bf16(__uint_as_float(w[i] << 16) * alpha, __uint_as_float(w[i] & 0xFFFF0000u) * alpha);
                __syncwarp();
                tmem_st32(t_s, w);
              }
              load32(x, first ? 64 : 0);
              if (!first) page(0, pa, pen_a, true);
              page(64, pb, pen_b, false);
              warm = __all_sync(kFull, m > -INFINITY);
            }
          } else {
            // Validity, visibility and penalty key by key, 32 keys at a time.  Keys from
            // `end` on are not seen; branch-free, as every lane has an end of its own.
            auto scores32 = [&](float (&s)[32], int c, auto timed) {
              const PageMeta& pg = c < 2 ? pa : pb;
              const float pen = c < 2 ? pen_a : pen_b;
              const int end = min(pg.live - (c & 1) * 32, lim - key0 - c * 32);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float q = decltype(timed)::value ? block_penalty_log2(tq, times[c * 32 + i], p) : pen;
                s[i] = i < end ? fmaf(s[i], pg.c, -q) : -INFINITY;
              }
            };
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const float vs = c < 2 ? pa.vs : pb.vs;
              float s[32];
              uint32_t pk[16];
              __syncwarp();
              tmem_ld32f(t_s + c * 32, s);
              tmem_landed(s);
              if (kPen && (c < 2 ? pa.mode : pb.mode) == 2) scores32(s, c, std::true_type{});
              else scores32(s, c, std::false_type{});
              const float top = top32(s);
              if (__any_sync(kFull, top > m + kRescaleThreshold)) {  // what is stored of this step follows the new maximum
                const float alpha = raise(top);
#pragma unroll 1
                for (int k = 0; k < c; ++k) {
                  uint32_t w[16];
                  __syncwarp();
                  tmem_ld16(t_s + k * 16, w);
                  tmem_landed(w);
#pragma unroll
                  for (int i = 0; i < 16; ++i)
                    w[i] = pack_bf16(__uint_as_float(w[i] << 16) * alpha, __uint_as_float(w[i] & 0xFFFF0000u) * alpha);
                  __syncwarp();
                  tmem_st16(t_s + k * 16, w);
                }
              }
              const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float e0 = ex2(s[i] - base), e1 = ex2(s[i + 1] - base);
                l += e0 + e1;
                // a scale that is not finite stays away from rows that do not see the key
                pk[i / 2] = pack_bf16(e0 == 0.0f ? 0.0f : e0 * vs, e1 == 0.0f ? 0.0f : e1 * vs);
              }
              __syncwarp();
              tmem_st16(t_s + c * 16, pk);
            }
            warm = __all_sync(kFull, m > -INFINITY);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + sub);
        }
        // ------------------------------------------------------- output
        if (ok) ok = wait_bar_all<kSuspend>(o_final, items & 1u, p, abort_flag);
        if (ok) {
          tc_fence_after();
          const bool whole = n == it.steps;
          const size_t at = (size_t)head * p.b.T + it.first + row;
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
          float* slot = whole ? nullptr : slot_of<D>(p, blockIdx.x, began ? 1 : 0);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float x[32];
            __syncwarp();
            tmem_ld32f(t_o + c * 32, x);
            tmem_landed(x);
            if (valid) {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 v = make_float4(x[i], x[i + 2], x[i + 1], x[i + 3]);
                if (whole) store_cols(p, at, c * 32 + i, v, inv);
                else *reinterpret_cast<float4*>(slot + pr * D + c * 32 + i) = v;
              }
            }
          }
          if (whole && valid) store_lse(p, at, m, l);
          if (!whole && valid) *reinterpret_cast<float2*>(slot + kTile * D + 2 * pr) = make_float2(m, l);
        }
        // a step left early may still have TMEM accesses in flight
        tmem_wait_st();
        tmem_wait_ld();
      }
    }
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
    while (next()) {
      // ------------------------------------------------- keys and values
      constexpr int kLoads = D / 16;  // 16-byte loads of a thread per K or V block
      const int w = warp - kWidenWarp, page_of = w >> 1;
      const int rlo = lane >> 2, ch = lane & 3;
      // load i: row 32 w + 8 (i / halves) + rlo, 16 codes at 64 (i % halves) + 16 ch
      uint4 kr[kLoads], vr[kLoads];
      // This warp's page of step j, -1 if it holds no valid key; its entry of the
      // page table is read a step before it is used.
      int page = -1, entry = -1;
      auto read_entry = [&](int j) {
        const int no = (step0 + j) * 2 + page_of;
        entry = -1;
        if (j < n && no * kBlock < it.len) entry = __ldg(p.b.page_table + (size_t)it.b * p.b.max_pages + no);
      };
      auto find_page = [&](int j) {
        const int no = (step0 + j) * 2 + page_of;
        page = entry;
        if (j < n && no * kBlock < it.len && (page < 0 || page >= p.c.n_pages)) {
          report(p.status, kStatusData);
          page = -1;
        }
        read_entry(j + 1);
      };
      auto load = [&](const int8_t* codes, uint4 (&x)[kLoads]) {
        const int8_t* src = codes + ((size_t)max(page, 0) * p.c.H + it.hk) * kBlock * D;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int row = (w & 1) * 32 + i / L::kHalves * 8 + rlo;
          x[i] = page < 0 ? make_uint4(0u, 0u, 0u, 0u)
                          : __ldg(reinterpret_cast<const uint4*>(src + row * D + i % L::kHalves * 64 + ch * 16));
        }
      };
      auto widen = [&](uint8_t* block, const uint4 (&x)[kLoads]) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int row = w * 32 + i / L::kHalves * 8 + rlo;
          uint8_t* dst = block + i % L::kHalves * L::kAtom + row * 128;
          *reinterpret_cast<uint4*>(dst + (((2 * ch) ^ (row & 7)) << 4)) =
              make_uint4(widen2(x[i].x), widen2(x[i].x >> 8), widen2(x[i].y), widen2(x[i].y >> 8));
          *reinterpret_cast<uint4*>(dst + (((2 * ch + 1) ^ (row & 7)) << 4)) =
              make_uint4(widen2(x[i].z), widen2(x[i].z >> 8), widen2(x[i].w), widen2(x[i].w >> 8));
        }
      };
      // the page's scales and times, one step ahead like its codes
      float ks = 0.0f, vs = 1.0f, t0 = NAN, t1 = NAN;
      auto load_meta = [&]() {
        ks = vs = 1.0f;
        t0 = t1 = NAN;
        if (page >= 0) {
          ks = __ldg(p.c.k_scale + (size_t)page * p.c.H + it.hk);
          vs = __ldg(p.c.v_scale + (size_t)page * p.c.H + it.hk);
          if (kPen) {
            t0 = __ldg(p.c.times + (size_t)page * kBlock + lane);
            t1 = __ldg(p.c.times + (size_t)page * kBlock + 32 + lane);
          }
        }
      };
      read_entry(0);
      find_page(0);
      load(p.c.k, kr);
      load(p.c.v, vr);
      load_meta();
      for (int j = 0; j < n; ++j) {
        const uint32_t q = done + j;
        const int s = q & 1, slot = q & 3;
        // keys of the page that rows may see: 0 for a page past the end or outside the cache
        const int live = page < 0 ? 0 : max(0, min(kBlock, it.len - ((step0 + j) * 2 + page_of) * kBlock));
        if ((w & 1) == 0) {
          PageMeta pm;
          pm.c = ks * p.scale_log2;
          pm.vs = vs;
          pm.lv = log2_approx(vs);
          pm.iv = rcp_approx(vs);
          pm.live = live;
          pm.mode = 0;
          pm.t = 0.0f;
          if (kPen) {
            // a key past the end counts as one without a time
            if (lane >= live) t0 = NAN;
            if (lane + 32 >= live) t1 = NAN;
            pm.t = __shfl_sync(kFull, t0, 0);
            if (__all_sync(kFull, t0 == pm.t && t1 == pm.t)) pm.mode = 1;
            else if (__any_sync(kFull, t0 == t0 || t1 == t1)) pm.mode = 2;
            float* times = reinterpret_cast<float*>(smem + L::kTimes) + slot * kStep + page_of * kBlock;
            times[lane] = t0;
            times[lane + 32] = t1;
          }
          pm.plain = live == kBlock && pm.mode != 2 && vs >= kScaleLow && vs <= kScaleHigh;
          if (lane == 0) reinterpret_cast<PageMeta*>(smem + L::kMeta)[2 * slot + page_of] = pm;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(m_full + slot);
        widen(smem + L::kK + s * L::kBlockBytes, kr);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full + s);
        find_page(j + 1);
        load(p.c.k, kr);
        load_meta();
        // Once the last step's scores are complete, the values of the step before it
        // are free, and its own keys.  (A tile's steps take two barriers in turn: this
        // step's scores may be complete as well by now, but not the next one's.)
        if (j > 0) {
          const uint32_t last = (subs == 2 ? done_b : done) + j - 1;
          if (!wait_bar_all<kSuspend>(s_full + 2 * (subs - 1) + (last & 1u), (last >> 1) & 1u, p, abort_flag)) break;
        }
        widen(smem + L::kV + s * L::kBlockBytes, vr);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && j == n - 1) mbar_arrive(v_full);  // else the next step's keys tell
        load(p.c.v, vr);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    while (next()) {
      if (warp != kMmaWarp) continue;
      // ------------------------------------------------------ MMA issuer
      constexpr uint32_t kIdescS = idesc_bf16_f32(128, kStep, 0, 0);
      constexpr uint32_t kIdescO = idesc_bf16_f32(128, D, 0, 1);
      // a descriptor's low bits hold the address / 16
      const uint64_t q_d = sw128_desc(smem_u32(smem + L::kQ), 16, 1024);
      const uint64_t k_d = sw128_desc(smem_u32(smem + L::kK), 16, 1024);
      const uint64_t v_d = sw128_desc(smem_u32(smem + L::kV), L::kAtom, 1024);
      auto issue_s = [&](int sub, int j) {
        const uint32_t k_buf = (done + j) & 1u, x = (sub ? done_b : done) + j;
#pragma unroll
        for (int kk = 0; kk < L::kHalves * 4; ++kk) {
          const uint32_t off = (kk >> 2) * L::kAtom + (kk & 3) * 32;
          umma_ss_one(tmem + (uint32_t)(128 * sub), q_d + ((sub * L::kBlockBytes + off) >> 4),
                  k_d + ((k_buf * L::kBlockBytes + off) >> 4), kIdescS, kk > 0 ? 1u : 0u);
        }
        umma_commit_one(s_full + 2 * sub + (x & 1u));
      };
      auto wait_k = [&](int j) {
        return wait_bar_all<kSuspend>(k_full + ((done + j) & 1u), ((done + j) >> 1) & 1u, p, abort_flag);
      };
      bool ok = wait_bar_all<kSuspend>(q_full, items & 1u, p, abort_flag) && wait_k(0);
      if (ok) {
        tc_fence_after();
        for (int sub = 0; sub < subs; ++sub) issue_s(sub, 0);
      }
      for (int j = 0; ok && j < n; ++j) {
        const uint32_t buf = (done + j) & 1u;
        const bool more = j + 1 < n;
        // the keys of the next step, and with them this step's values: a widening
        // warp stores the values of a step before the keys of the next
        ok = more ? wait_k(j + 1) : wait_bar_all<kSuspend>(v_full, items & 1u, p, abort_flag);
        for (int sub = 0; ok && sub < subs; ++sub) {
          ok = wait_bar_all<kSuspend>(p_full + sub, ((sub ? done_b : done) + j) & 1u, p, abort_flag);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kStep / 16; ++kk)
            umma_ts_one(tmem + kTmemO + (uint32_t)(D * sub), tmem + (uint32_t)(128 * sub + 8 * kk),
                    v_d + ((buf * L::kBlockBytes + kk * 2048) >> 4), kIdescO, j > 0 || kk > 0 ? 1u : 0u);
          if (more) issue_s(sub, j + 1);
        }
      }
      umma_commit_one(o_final);
    }
  }

  if (warp == kMmaWarp) {  // all issued MMAs complete before TMEM is released
    umma_commit_one(drain);
    drain_wait(drain, 0, p);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the items that several blocks share: blocks (x, y) look at the border
// between the stretches x and x + 1 and join the item that lies across it, if it
// is that item's first border; y takes 32 of its pairs.  The item, and the slots
// that hold parts of it, are found by one warp; a thread then takes 4 columns of
// several pairs, all their loads of a slot issued together.
constexpr int kJoinThreads = 256, kJoinPairs = 32;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_tiles_kernel(const CacheAttnParams p) {
  constexpr int kEach = kJoinPairs * (D / 4) / kJoinThreads;  // pairs of a thread
  __shared__ Item item;
  __shared__ int parts, slots[kGrid];
  const int tid = threadIdx.x, lane = tid & 31;
  const long long total = p.base[p.b.B], share = share_of(total);
  const int c0 = (int)blockIdx.x;
  const long long u = (c0 + 1) * share;
  if (u >= total) {
    wait_dependency();
    return;
  }
  if (tid < 32) {
    const Item it = find_item(p, u);
    int n = 0;
    if (it.start < u && it.start >= c0 * share && it.pairs > (int)blockIdx.y * kJoinPairs) {
      // a block whose stretch touches the item without a step of it has written nothing
      const long long end = it.start + it.units();
      for (int c = c0; c * share < end; c += 32) {
        const long long from = (c + lane) * share;
        const bool has = from < end && it.step(from + share) > it.step(from);
        const unsigned who = __ballot_sync(kFull, has);
        if (has) slots[n + __popc(who & ((1u << lane) - 1u))] = 2 * (c + lane) + (c + lane == c0 ? 1 : 0);
        n += __popc(who);
      }
    }
    if (lane == 0) {
      item = it;
      parts = n;
    }
  }
  __syncthreads();
  wait_dependency();
  const int n = parts;
  if (n < 2) return;  // not the item's first border, or one block has all of it
  const Item it = item;
  const int col = tid % (D / 4) * 4, r0 = blockIdx.y * kJoinPairs + tid / (D / 4);
  float mm[kEach], ll[kEach];
  float4 sum[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    mm[e] = -INFINITY;
    ll[e] = 0.0f;
    sum[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  for (int k = 0; k < n; ++k) {
    const float* slot = p.partial + (size_t)slots[k] * (kTile * (D + 2));
    float2 x[kEach];
    float4 y[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int r = r0 + e * (kJoinThreads / (D / 4));
      if (r < it.pairs) {
        x[e] = *reinterpret_cast<const float2*>(slot + kTile * D + 2 * r);
        y[e] = *reinterpret_cast<const float4*>(slot + r * D + col);
      }
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      if (r0 + e * (kJoinThreads / (D / 4)) >= it.pairs) continue;
      const float mn = fmaxf(mm[e], x[e].x), base = mn == -INFINITY ? 0.0f : mn;
      const float a = ex2(mm[e] - base), w = ex2(x[e].x - base);
      mm[e] = mn;
      ll[e] = ll[e] * a + w * x[e].y;
      sum[e].x = sum[e].x * a + w * y[e].x, sum[e].y = sum[e].y * a + w * y[e].y;
      sum[e].z = sum[e].z * a + w * y[e].z, sum[e].w = sum[e].w * a + w * y[e].w;
    }
  }
  const int i0 = (int)(it.pair0 / p.group), g0 = (int)(it.pair0 - (long long)i0 * p.group);
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int r = r0 + e * (kJoinThreads / (D / 4));
    if (r >= it.pairs) continue;
    const int i = (int)((unsigned)(g0 + r) / (unsigned)p.group), g = g0 + r - i * p.group;
    const size_t at = (size_t)(it.hk * p.group + g) * p.b.T + it.first + i0 + i;
    store_cols(p, at, col, sum[e], ll[e] == 0.0f ? 0.0f : 1.0f / ll[e]);
    if (col == 0) store_lse(p, at, mm[e], ll[e]);
  }
}

template <int D>
cudaError_t launch_t(const CacheAttnParams& p, cudaStream_t stream) {
  constexpr int bytes = TilesLayout<D>::kBytes;
  const bool limit = p.wait_polls != kNoPollLimit;
  auto kernel = p.q_times != nullptr ? limit ? tiles_kernel<D, true, false> : tiles_kernel<D, true, true>
                                     : limit ? tiles_kernel<D, false, false> : tiles_kernel<D, false, true>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  plan_kernel<<<1, 1024, 0, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = launch_after(kernel, dim3(kGrid), kThreads, bytes, stream, p)) != cudaSuccess) return e;
  return launch_after(join_tiles_kernel<D>, dim3(kGrid - 1, kTile / kJoinPairs), kJoinThreads, 0, stream, p);
}

}  // namespace

size_t cache_tiles_partial_bytes(int d) { return (size_t)2 * kGrid * kTile * (d + 2) * sizeof(float); }

cudaError_t launch_cache_tiles(const CacheAttnParams& p, cudaStream_t stream) {
  return p.c.d == 64 ? launch_t<64>(p, stream) : launch_t<128>(p, stream);
}

}  // namespace h3
