// C ABI of the paged int8 cache: argument validation, workspace layout and
// launches.  See the cache section of include/h3attn.h for the contract.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "cache.cuh"
#include "h3attn.h"

namespace {

constexpr size_t kStatusBytes = 256;

bool misaligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

int check_cache(const h3attn_cache* c, h3::CacheRef* out) {
  if (c == nullptr || c->n_pages < 1 || c->H < 1 || c->H > 65535) return H3ATTN_EINVAL;
  if (!(c->d == 64 || c->d == 128) || c->block != h3::kBlock) return H3ATTN_EUNSUPPORTED;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return H3ATTN_EINVAL;
  if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->k_scale, 4) || misaligned(c->v_scale, 4) ||
      misaligned(c->times, 16))
    return H3ATTN_EALIGN;
  *out = h3::CacheRef{c->n_pages, c->H, c->d, c->k, c->v, c->k_scale, c->v_scale, c->times};
  return H3ATTN_OK;
}

int check_batch(const h3attn_batch* b, h3::BatchRef* out) {
  if (b == nullptr || b->B < 1 || b->T < 0 || b->max_pages < 1) return H3ATTN_EINVAL;
  // Positions and packed rows are 32-bit, with room for a tile past the end.  Each block finds
  // its rows by a scan over the sequences (140 take a microsecond; appending a token of each of
  // 65,536 takes 35 ms), so B is bounded: 2^24 sequences would hold the GPU for half an hour.
  if (b->T > (1 << 30) || b->B > (1 << 16) || b->max_pages > (1 << 24)) return H3ATTN_EUNSUPPORTED;
  if (!b->row_start || !b->length || !b->page_table) return H3ATTN_EINVAL;
  if (misaligned(b->row_start, 4) || misaligned(b->length, 4) || misaligned(b->page_table, 4)) return H3ATTN_EALIGN;
  *out = h3::BatchRef{b->B, b->T, b->max_pages, b->row_start, b->length, b->page_table};
  return H3ATTN_OK;
}

// a [heads][rows][d] tensor by strides: 16-byte pieces of a row are read whole
int check_strided(const void* p, int64_t head, int64_t row) {
  if (p == nullptr || head < 0 || row < 0) return H3ATTN_EINVAL;
  return misaligned(p, 16) || head % 8 != 0 || row % 8 != 0 ? H3ATTN_EALIGN : H3ATTN_OK;
}

int check_ws(const void* ws, size_t have, size_t need) {
  if (ws == nullptr || have < need) return H3ATTN_EWORKSPACE;
  return misaligned(ws, 16) ? H3ATTN_EALIGN : H3ATTN_OK;
}

bool finite_nonneg(float x) { return std::isfinite(x) && x >= 0.0f; }

// Up to this many (query row, head of the group) pairs of a sequence go through
// the kernel for few rows.  There / in tensor-core tiles, us, with 32 pairs, then 40:
// 2 sequences of 16,384 rows, 16 heads of 128, 69 / 83, 97 / 82; one of 57,402, 8 heads,
// 60 / 81, 85 / 81; 32 of 4,000, 8 heads, 125 / 152, 172 / 153; 8 of 2,000, 16 heads of
// 64, 29 / 42, 38 / 43; one of 2,079, 56 heads of 128, 32 / 40, 36 / 41.
constexpr long long kFewPairs = 32;

// status word | the tile kernel's line [B + 1] | partial results.  A batch whose
// rows all fit the kernel for few rows needs no line.
struct ForwardLayout {
  size_t base, partial, total;
};
ForwardLayout forward_layout(int H, int Hkv, int d, int T, int B) {
  const long long pairs = (long long)T * (H / Hkv);
  ForwardLayout l;
  l.base = kStatusBytes;
  l.partial = l.base;
  size_t partial = h3::cache_rows_partial_bytes(d, pairs);
  if (pairs > kFewPairs) {
    l.partial += ((size_t)(B + 1) * sizeof(long long) + 255) / 256 * 256;
    const size_t tiles = h3::cache_tiles_partial_bytes(d);
    if (tiles > partial) partial = tiles;
  }
  l.total = l.partial + partial;
  return l;
}

}  // namespace

extern "C" {

size_t h3attn_cache_workspace_bytes(const h3attn_cache* cache, int H, int T, int B) {
  if (cache == nullptr || cache->H < 1 || H < 1 || H % cache->H != 0 || T < 0 || B < 1) return 0;
  if (!(cache->d == 64 || cache->d == 128)) return 0;
  return forward_layout(H, cache->H, cache->d, T, B).total;
}

int h3attn_cache_append(const h3attn_cache* cache, const h3attn_batch* batch, const uint16_t* k, int64_t k_head_stride,
                        int64_t k_row_stride, const uint16_t* v, int64_t v_head_stride, int64_t v_row_stride,
                        const h3attn_rope* rope, const float* row_times, void* ws, size_t ws_bytes, void* stream) {
  h3::AppendParams p{};
  if (int rc = check_cache(cache, &p.c)) return rc;
  if (int rc = check_batch(batch, &p.b)) return rc;
  if (p.b.T == 0) return H3ATTN_OK;
  if (int rc = check_strided(k, k_head_stride, k_row_stride)) return rc;
  if (int rc = check_strided(v, v_head_stride, v_row_stride)) return rc;
  if (rope != nullptr) {
    if (!rope->cos || !rope->sin || rope->n_pos < 1 || rope->dim < 16 || rope->dim > p.c.d || rope->dim % 16 != 0)
      return H3ATTN_EINVAL;
    if (misaligned(rope->cos, 16) || misaligned(rope->sin, 16) || misaligned(rope->index, 4)) return H3ATTN_EALIGN;
    p.rope = h3::RopeRef{rope->cos, rope->sin, rope->index, rope->n_pos, rope->dim, rope->interleaved};
  }
  if (row_times != nullptr && p.c.times == nullptr) return H3ATTN_EINVAL;
  if (misaligned(row_times, 4)) return H3ATTN_EALIGN;
  if (int rc = check_ws(ws, ws_bytes, kStatusBytes)) return rc;
  p.k = k;
  p.v = v;
  p.k_head = k_head_stride;
  p.k_row = k_row_stride;
  p.v_head = v_head_stride;
  p.v_row = v_row_stride;
  p.row_times = row_times;
  p.minus_zero = -0.0f;
  p.status = static_cast<int*>(ws);
  return h3::launch_cache_append(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? H3ATTN_OK : H3ATTN_ECUDA;
}

int h3attn_cache_read(const h3attn_cache* cache, const h3attn_batch* batch, uint16_t* k, uint16_t* v, void* ws,
                      size_t ws_bytes, void* stream) {
  h3::ReadParams p{};
  if (int rc = check_cache(cache, &p.c)) return rc;
  if (int rc = check_batch(batch, &p.b)) return rc;
  if (p.b.T == 0) return H3ATTN_OK;
  if (k == nullptr && v == nullptr) return H3ATTN_EINVAL;
  if (misaligned(k, 16) || misaligned(v, 16)) return H3ATTN_EALIGN;
  if (int rc = check_ws(ws, ws_bytes, kStatusBytes)) return rc;
  p.k = k;
  p.v = v;
  p.status = static_cast<int*>(ws);
  return h3::launch_cache_read(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? H3ATTN_OK : H3ATTN_ECUDA;
}

int h3attn_cache_forward(const h3attn_cache* cache, const h3attn_batch* batch, int H, int max_rows, const uint16_t* q,
                         int64_t q_head_stride, int64_t q_row_stride, int causal, const h3attn_penalty* pen,
                         const float* q_times, uint16_t* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
  h3::CacheAttnParams p{};
  if (int rc = check_cache(cache, &p.c)) return rc;
  if (int rc = check_batch(batch, &p.b)) return rc;
  if (H < 1 || H > 65535 || H % p.c.H != 0 || max_rows < 0) return H3ATTN_EINVAL;
  if (pen != nullptr) {
    if (!finite_nonneg(pen->strength) || !finite_nonneg(pen->window) || !finite_nonneg(pen->cap) ||
        !std::isfinite(pen->falloff))
      return H3ATTN_EINVAL;
    if (pen->strength > 0.0f && pen->cap > 0.0f) {
      if (!(pen->falloff > 0.0f) || q_times == nullptr || p.c.times == nullptr) return H3ATTN_EINVAL;
      if (misaligned(q_times, 4)) return H3ATTN_EALIGN;
      const float log2e = 1.4426950408889634f;
      p.q_times = q_times;
      p.window = pen->window;
      // An infinite factor would make 0 inf of a key inside the window.  A penalty of 2^26
      // (log2 units) leaves nothing of a key beside one without, for scores lie within 2^24;
      // maxima of masked keys then still have an ulp of 8, far inside the kernels' margins.
      p.inv_falloff = std::min(1.0f / pen->falloff, FLT_MAX);
      p.strength_log2 = std::min(pen->strength * log2e, FLT_MAX);
      p.cap_log2 = std::min(pen->cap * log2e, 67108864.0f);
    }
  }
  if (p.b.T == 0) return H3ATTN_OK;
  if (int rc = check_strided(q, q_head_stride, q_row_stride)) return rc;
  if (o == nullptr) return H3ATTN_EINVAL;
  if (misaligned(o, 16) || misaligned(lse, 4)) return H3ATTN_EALIGN;
  const ForwardLayout lay = forward_layout(H, p.c.H, p.c.d, p.b.T, p.b.B);
  if (int rc = check_ws(ws, ws_bytes, lay.total)) return rc;
  p.H = H;
  p.group = H / p.c.H;
  p.causal = causal != 0;
  p.q = q;
  p.q_head = q_head_stride;
  p.q_row = q_row_stride;
  p.o = o;
  p.lse = lse;
  p.status = static_cast<int*>(ws);
  p.scale_log2 = 1.4426950408889634f / std::sqrt((float)p.c.d);
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  p.base = reinterpret_cast<long long*>(wsb + lay.base);
  p.partial = reinterpret_cast<float*>(wsb + lay.partial);
  p.wait_polls = h3::wait_poll_limit();
  p.wait_ns = h3::wait_time_limit_ns();
  const long long pairs = (long long)(max_rows > 0 && max_rows < p.b.T ? max_rows : p.b.T) * p.group;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = pairs <= kFewPairs ? h3::launch_cache_rows(p, pairs, st) : h3::launch_cache_tiles(p, st);
  return e == cudaSuccess ? H3ATTN_OK : H3ATTN_ECUDA;
}

}  // extern "C"
