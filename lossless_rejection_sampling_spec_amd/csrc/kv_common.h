// kv_common.h -- what the cache kernels share: the page layout, the request
// rules and small wave helpers.
//
// A page of one layer holds, per KV head, one unit of P tokens of dimension D
// (include/specverify.h states the layout as the ABI's):
//   K codes   [P][D/2]             a token's dims in order, two codes per byte
//   V codes   [P/8][16][8][D/32]   8 tokens side by side for each 16th of D
//   K scales  [P/8][D/32][8]       8 tokens side by side for each 32 dims
//   V scales  [P/8][D/32][8]
// The layout is that of the matrix instructions' operands: a lane's K operand
// is D/8 contiguous bytes of one token, its V operand D/4 contiguous bytes
// (its 16th of the dims for 8 tokens), its 8 scales one 64-bit word, so the
// attention loads operands straight into registers and never goes through LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "specverify.h"

namespace svk {

constexpr int MAX_BATCH = 1024;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Bytes of one unit (page x KV head).
__host__ __device__ constexpr int64_t unit_bytes(int page, int d) {
  return (int64_t)page * (d + d / 16);
}
__host__ __device__ constexpr int off_v(int page, int d) { return page * d / 2; }
__host__ __device__ constexpr int off_ks(int page, int d) { return page * d; }
__host__ __device__ constexpr int off_vs(int page, int d) { return page * d + page * d / 32; }

inline bool dim_ok(int d) { return d == 64 || d == 128 || d == 256; }
inline bool page_ok(int p) { return p >= 16 && p <= 256 && (p & (p - 1)) == 0; }
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

template <typename V>
__device__ __forceinline__ V load_any(const void* p) {   // no alignment beyond the element's
  V v;
  __builtin_memcpy(&v, p, sizeof(V));
  return v;
}

// The first request whose offsets break the packing rule (negative, going
// back, or past total_rows), `batch` if none does: that request and every
// later one are BAD_K.  One wave, all lanes active; every lane gets the answer.
__device__ __forceinline__ int first_broken(const int32_t* cu, int batch, int total_rows) {
  const int lane = threadIdx.x & 63;
  for (int b0 = 0; b0 < batch; b0 += 512) {
    int c0[8], c1[8];                          // (the loads of 512 requests go out together)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int b = min(b0 + 64 * i + lane, batch - 1);
      c0[i] = cu[b];
      c1[i] = cu[b + 1];
      if (b0 + 64 * (i + 1) >= batch) break;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int b = b0 + 64 * i + lane;
      const bool bad = b < batch && (c0[i] < 0 || c1[i] < c0[i] || c1[i] > total_rows);
      const unsigned long long m = __ballot(bad);
      if (m) return b0 + 64 * i + __builtin_ctzll(m);
      if (b0 + 64 * (i + 1) >= batch) break;
    }
  }
  return batch;
}

}  // namespace svk
