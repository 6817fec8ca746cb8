// What the two attention kernels over the paged int8 cache share.
#pragma once
#include <cstdint>

#include "cache.cuh"
#include "softmax.cuh"

namespace h3 {

// Widening codes to bf16 exactly: with 0x43 in front, the low 7 bits of a code
// read as 128 + low in bf16 (ulp 1) and its sign bit alone as 128 or 256; their
// difference is the code.  Two logic operations and one packed subtraction give
// the codes in bytes 0 and 2 of w as two bf16.
__device__ __forceinline__ uint32_t widen2(uint32_t w) {
  uint32_t lo, hi, r;
  asm("lop3.b32 %0, %1, 0x007F007F, 0x43004300, 0xEA;" : "=r"(lo) : "r"(w));  // (w & a) | b
  asm("lop3.b32 %0, %1, 0x00800080, 0x43004300, 0xEA;" : "=r"(hi) : "r"(w));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(lo), "r"(hi));
  return r;
}


// 32 columns of the warp's TMEM lanes as floats; the values are there after tmem_landed(r).
__device__ __forceinline__ void tmem_ld32f(uint32_t taddr, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
        "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
        "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr));
}
// Waits for the thread's TMEM loads; no use of r is scheduled before it.
__device__ __forceinline__ void tmem_landed(float (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]),
                 "+f"(r[7]), "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]),
                 "+f"(r[14]), "+f"(r[15]), "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]),
                 "+f"(r[21]), "+f"(r[22]), "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]),
                 "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])
               :
               : "memory");
}

// Columns [col, col + 4) of a pair's row of the output, and its LSE: the pair
// (query row, head of the group) is number `pair` in the list of the sequence
// whose packed rows begin at `first`; v unnormalised, m in log2 units.
__device__ __forceinline__ void store_cols(const CacheAttnParams& p, int first, int hk, long long pair, int col,
                                           float4 v, float m, float l) {
  const int i = (int)(pair / p.group), h = hk * p.group + (int)(pair % p.group);
  const size_t at = (size_t)h * p.b.T + first + i;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  *reinterpret_cast<uint2*>(p.o + at * p.c.d + col) =
      make_uint2(sm::pack_bf16(v.x * inv, v.y * inv), sm::pack_bf16(v.z * inv, v.w * inv));
  if (p.lse != nullptr && col == 0) p.lse[at] = (m + log2f(l)) * sm::kLn2;
}

}  // namespace h3
