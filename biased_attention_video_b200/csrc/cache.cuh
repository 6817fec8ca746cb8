// Paged int8 cache of keys and values: what its kernels share.  See the cache
// section of include/h3attn.h for the layout and the quantisation rule.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "kernels.cuh"

namespace h3 {

constexpr float kMinScale = 7.888609052210118e-31f;  // 2^-100, the smallest scale a block takes

// h3attn_cache
struct CacheRef {
  int n_pages, H, d;
  int8_t *k, *v;            // [n_pages][H][64][d]
  float *k_scale, *v_scale; // [n_pages][H]
  float* times;             // [n_pages][64] or null
};

// h3attn_batch: rows [row_start[b], row_start[b + 1]) of T packed rows belong to sequence b
struct BatchRef {
  int B, T, max_pages;
  const int32_t* row_start;   // [B + 1]
  const int32_t* length;      // [B]
  const int32_t* page_table;  // [B][max_pages]
};

struct RopeRef {
  const float *cos, *sin;  // [n_pos][dim / 2]; null: no rotation
  const int32_t* index;    // [T] or null (the row's position)
  int n_pos, dim, interleaved;
};

struct AppendParams {
  CacheRef c;
  BatchRef b;
  RopeRef rope;
  const uint16_t *k, *v;
  long long k_head, k_row, v_head, v_row;  // strides in elements
  const float* row_times;
  int* status;
  float minus_zero;  // -0, see mul2_rn
};
cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t stream);

struct ReadParams {
  CacheRef c;
  BatchRef b;
  uint16_t *k, *v;  // [H][T][d] or null
  int* status;
};
cudaError_t launch_cache_read(const ReadParams& p, cudaStream_t stream);

struct CacheAttnParams {
  CacheRef c;
  BatchRef b;
  int H, group, causal;  // query heads, query heads of one K/V head
  const uint16_t* q;
  long long q_head, q_row;
  const float* q_times;  // null: no penalty
  uint16_t* o;           // [H][T][d]
  float* lse;            // [H][T] or null
  int* status;
  float scale_log2;      // log2(e) / sqrt(d)
  float window, inv_falloff, strength_log2, cap_log2;
  float* partial;        // partial results (see the kernels)
  long long* base;       // [B + 1], the tile kernel's line (see cache_tiles.cu)
  uint32_t wait_polls;   // bounded waits of the tile kernel
  uint64_t wait_ns;
};

// Few rows per sequence; see cache_rows.cu.  pairs: most (query row, head of the
// group) pairs of one sequence.
size_t cache_rows_partial_bytes(int d, long long pairs);
cudaError_t launch_cache_rows(const CacheAttnParams& p, long long pairs, cudaStream_t stream);

// Tensor-core tiles of 256 pairs; see cache_tiles.cu.
size_t cache_tiles_partial_bytes(int d);
cudaError_t launch_cache_tiles(const CacheAttnParams& p, cudaStream_t stream);

// ------------------------------------------------------------ device side

// Rows [first, first + n) of sequence b in the packed rows, forced into [0, T]
// (offsets that are not ascending in [0, T] are reported).
struct SeqRows {
  int first, n;
};
__device__ __forceinline__ SeqRows seq_rows(const BatchRef& r, int b, int* status) {
  const int a = __ldg(r.row_start + b), e = __ldg(r.row_start + b + 1);
  const int first = min(max(a, 0), r.T), last = min(max(e, first), r.T);
  if (first != a || last != e) report(status, kStatusData);
  return SeqRows{first, last - first};
}

// Cached rows of sequence b, forced into what its row of the page table holds.
__device__ __forceinline__ int seq_length(const BatchRef& r, int b, int* status) {
  const int n = __ldg(r.length + b);
  const int held = min(max(n, 0), r.max_pages * kBlock);
  if (held != n) report(status, kStatusData);
  return held;
}

// Piece x of the call: the rows of one sequence that lie in one page.  Pieces
// are counted sequence by sequence; sequence b's rows take the positions from
// length[b] on.  b = -1 when the call has no piece x.
struct Piece {
  int b, page_no, lo, hi;  // positions [lo, hi) of sequence b, inside its page page_no
  int row;                 // packed row of position lo
  int held;                // earlier rows of the page that stay
};
// Every warp finds the piece for itself (no barrier): a lane counts the pieces of
// kSeqs consecutive sequences, all their loads issued together.
__device__ __forceinline__ Piece find_piece(const BatchRef& r, int x, int* status) {
  constexpr int kSeqs = 4;
  const int lane = threadIdx.x & 31;
  Piece p{};
  p.b = -1;
  int base = 0;
  for (int b0 = 0; b0 < r.B && p.b < 0; b0 += 32 * kSeqs) {
    int start[kSeqs], n[kSeqs], first[kSeqs], cnt[kSeqs], mine = 0;
#pragma unroll
    for (int e = 0; e < kSeqs; ++e) {
      const int b = b0 + lane * kSeqs + e;
      start[e] = n[e] = first[e] = cnt[e] = 0;
      if (b < r.B) {
        const SeqRows s = seq_rows(r, b, status);
        start[e] = seq_length(r, b, status);
        first[e] = s.first;
        n[e] = min(s.n, r.max_pages * kBlock - start[e]);
        if (n[e] < s.n) report(status, kStatusData);
        cnt[e] = n[e] > 0 ? (start[e] + n[e] - 1) / kBlock - start[e] / kBlock + 1 : 0;
      }
      mine += cnt[e];
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    int i = x - base - (incl - mine);  // the piece's number among this lane's
    const unsigned who = __ballot_sync(0xFFFFFFFFu, i >= 0 && i < mine);
    if (who != 0u) {
      const int from = __ffs(who) - 1;
      int e_at = 0, s_at = 0, n_at = 0, f_at = 0;
#pragma unroll
      for (int e = kSeqs - 1; e >= 0; --e) {  // the last sequence whose pieces begin at or before i
        int before = 0;
#pragma unroll
        for (int k = 0; k < e; ++k) before += cnt[k];
        if (i >= before && i < before + cnt[e]) {
          e_at = e;
          s_at = start[e];
          n_at = n[e];
          f_at = first[e];
          i -= before;
          break;
        }
      }
      p.b = b0 + from * kSeqs + __shfl_sync(0xFFFFFFFFu, e_at, from);
      const int begin = __shfl_sync(0xFFFFFFFFu, s_at, from);
      const int end = begin + __shfl_sync(0xFFFFFFFFu, n_at, from);
      p.page_no = begin / kBlock + __shfl_sync(0xFFFFFFFFu, i, from);
      p.lo = max(begin, p.page_no * kBlock);
      p.hi = min(end, (p.page_no + 1) * kBlock);
      p.row = __shfl_sync(0xFFFFFFFFu, f_at, from) + p.lo - begin;
      p.held = p.lo - p.page_no * kBlock;
    }
    base += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  return p;
}
// an upper bound of the pieces, known without the device arrays: a sequence of
// n rows lies in at most min(n, n / 64 + 2) pages
inline unsigned max_pieces(const BatchRef& r) {
  const long long a = r.T, b = (long long)r.T / kBlock + 2ll * r.B;
  return (unsigned)(a < b ? a : b);
}

// Page id of a sequence's page page_no, or -1 (reported) if the table holds none of the cache's pages.
__device__ __forceinline__ int page_id(const CacheRef& c, const BatchRef& r, int b, int page_no, int* status) {
  const int id = __ldg(r.page_table + (size_t)b * r.max_pages + page_no);
  if (id < 0 || id >= c.n_pages) {
    report(status, kStatusData);
    return -1;
  }
  return id;
}

}  // namespace h3
