// kvcache.hip -- the 4-bit paged KV cache around the verify
// (include/specverify.h states each operator):
//   spec_kv_append    head norms, rotation and quantisation of the call's rows
//                     (spec_kv_append_at of specverify_cache.h: at slots that are not
//                     positions)
//   spec_kv_reserve   pages for the rows of a call, copy-on-write of shared tails
//   spec_kv_release   positions given back after the drain
//   spec_kv_fork      sequences that share another one's pages
//   spec_kv_compact   live pages moved to the front of the pool
//
// Page state is the reference count alone: a page is free when its count is 0.
// Counts change by integer atomics only, so their values do not depend on the
// order; pages are handed out lowest id first.  Every result is deterministic.

#include "kv_common.h"

namespace svk {

// ------------------------------------------------------------------- append
//
// One head of one row is D/8 lanes, 8 dims each, so its sum of squares and the
// rotation's partner dims come by shuffles inside the head and a block of 32
// dims is four neighbouring lanes.  All arithmetic is fp64 and rounds once at
// the end: a code next to a border, or a bf16 query, then never depends on how
// the sum was ordered, and the same row gives the same bytes whichever call
// wrote it.  448 rows of 32 + 2 * 8 heads of D=128 take 10 us (12 MB: start and
// latency of the dependent loads), 9,300 rows 64 us (242 MB, 3.8 TB/s; the vector
// units are busy 90 % of that).

struct AppendArgs {
  const void *q, *k, *v;
  int64_t ld_q, ld_k, ld_v;
  const float *qw, *kw;
  float eps;
  const float* cos_sin;
  int max_position, rot, interleaved;
  const int32_t *cu, *ctx;
  const int32_t* offsets;       // added to a request's positions in the angles' table, or NULL
  int batch, total_rows, heads, kv_heads;
  uint8_t* pages;
  int64_t num_pages;
  int page, page_log2;
  const int32_t* table;
  int64_t ld_table;
  void* q_out;
  int64_t ld_qout;
  void *k_val, *v_val;
  int32_t* status;
  int data_blocks;
  int tasks, slices, slice_groups;   // waves' shares: rows * slices of the rows' head groups
};

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xf, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, false));
}
// lane ^ 1, lane ^ 2, and the mirrors of 8 and 16 lanes, which reach the other half
// once the lanes of a half agree
constexpr int DPP_XOR1 = 0xb1, DPP_XOR2 = 0x4e, DPP_MIRROR8 = 0x141, DPP_MIRROR16 = 0x140;

__device__ __forceinline__ double shfl_xor_f64(double x, int m) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)u, m);
  const uint32_t hi = (uint32_t)__shfl_xor((int)(uint32_t)(u >> 32), m);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double shfl_f64(double x, int src) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)u, src);
  const uint32_t hi = (uint32_t)__shfl((int)(uint32_t)(u >> 32), src);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// x as a float that a further rounding to 18 bits or fewer treats as x itself: the
// 20 mantissa bits of its upper word, the last one set if anything follows (rounding
// to odd), so that x lands on no tie or border that it is not on.
__device__ __forceinline__ float odd_f32(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t hi = (uint32_t)(u >> 32) | min((uint32_t)u, 1u);
  return (float)__builtin_bit_cast(double, (uint64_t)hi << 32);
}

// 1 / sqrt(s): the hardware's estimate and two steps of Newton's method (the first
// brings its error to about 2^-45, the second to fp64's own).
__device__ __forceinline__ double rsqrt_f64(double s) {
  double r = __builtin_amdgcn_rsq(s);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const double e = __builtin_fma(-s * r, r, 1.0);
    r = __builtin_fma(r * e, 0.5, r);
  }
  return s < __builtin_inf() ? r : 1.0 / s;    // 0 at infinity, NaN for NaN
}

// 8 codes, the first in the lowest four bits, nearest with ties to the even code.
__device__ __forceinline__ uint32_t pack_codes(const float* z) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, z[0], z[1], 1.f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, z[2], z[3], 1.f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, z[4], z[5], 1.f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, z[6], z[7], 1.f, 3);
}

template <typename T>
__device__ __forceinline__ T round_to(double x);
template <>
__device__ __forceinline__ float round_to<float>(double x) { return (float)x; }
template <>
__device__ __forceinline__ __bf16 round_to<__bf16>(double x) { return (__bf16)odd_f32(x); }

// Requests 8 dims of head hh of a row's q, k and v (past the last head: that one).
template <int D, typename T>
__device__ __forceinline__ void ask_head(T* raw, const T* qrow, const T* krow, const T* vrow, int hh,
                                         int c, int heads, int kv_heads) {
  hh = min(hh, heads + 2 * kv_heads - 1);
  const bool q = hh < heads, k = hh < heads + kv_heads;
  const T* src = q ? qrow : k ? krow : vrow;
  const int at = hh - (q ? 0 : k ? heads : heads + kv_heads);
  __builtin_memcpy(raw, src + (uint32_t)(at * D + 8 * c), 8 * sizeof(T));
}

template <int D, typename T>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 4 : D == 256 ? 2 : 3) void k_append(AppendArgs a) {
  constexpr int LPH = D / 8;                  // lanes per head
  constexpr int HPW = 64 / LPH;               // heads of a wave
  __shared__ int32_t scu[MAX_BATCH + 1], sctx[MAX_BATCH];
  __shared__ double sw[2][D];                 // the norms' weights
  __shared__ int sbroken;
  const int tid = threadIdx.x, lane = tid & 63;

  if ((int)blockIdx.x >= a.data_blocks) {     // statuses: a wave per request
    const int broken = first_broken(a.cu, a.batch, a.total_rows);
    const int b = ((int)blockIdx.x - a.data_blocks) * 4 + (tid >> 6);
    if (b >= a.batch) return;
    int st = SV_ROW_BAD_K;
    if (b < broken && a.cu[b + 1] > a.cu[b]) {
      const int rows = a.cu[b + 1] - a.cu[b], ctx = a.ctx[b], off = a.offsets ? a.offsets[b] : 0;
      st = SV_ROW_OK;
      if (ctx < 0 || off < 0 || (int64_t)ctx + off + rows > a.max_position) st = SV_ROW_BAD_PARAM;
      else {
        bool bad = false;
        const int s1 = (ctx + rows - 1) >> a.page_log2;
        for (int s = (ctx >> a.page_log2) + lane; s <= s1; s += 64)
          bad |= s >= a.ld_table ||
                 (uint32_t)a.table[(int64_t)b * a.ld_table + s] >= (uint64_t)a.num_pages;
        if (__any(bad)) st = SV_ROW_BAD_PAGE;
      }
    }
    if (lane == 0) a.status[b] = st;
    return;
  }

  if (tid == 0) sbroken = a.batch;
  for (int i = tid; i < D; i += 256) {
    sw[0][i] = a.qw ? (double)a.qw[i] : 1.0;
    sw[1][i] = a.kw ? (double)a.kw[i] : 1.0;
  }
  __syncthreads();
  for (int i = tid; i < a.batch; i += 256) {
    const int c0 = a.cu[i], c1 = a.cu[i + 1];
    scu[i] = c0;
    sctx[i] = a.ctx[i];
    if (i == a.batch - 1) scu[a.batch] = c1;
    if (c0 < 0 || c1 < c0 || c1 > a.total_rows) atomicMin(&sbroken, i);
  }
  __syncthreads();
  const int broken = sbroken;
  const int per_row = a.heads + 2 * a.kv_heads;
  const int c = tid % LPH;                    // dims 8c .. 8c+7 of the lane's head
  const int half = a.rot / 2;
  const bool second = 8 * c >= half, in_rot = 8 * c < a.rot;
  const int partner = lane + (in_rot ? (second ? -half / 8 : half / 8) : 0);

  // a wave takes a row's groups of HPW heads, or a slice of them where rows are few:
  // what belongs to the row is found once and stays scalar
  const int wave0 = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int task = wave0; task < a.tasks; task += a.data_blocks * 4) {
    const int row = task / a.slices, slice = task - row * a.slices;
    // its request: the last with cu[b] <= row (good up to `broken`)
    int lo = 0, hi = broken;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__builtin_amdgcn_readfirstlane(scu[mid + 1]) <= row) lo = mid + 1;
      else hi = mid;
    }
    if (lo >= broken) continue;
    const int b = lo, row0 = __builtin_amdgcn_readfirstlane(scu[b]);
    const int ctx = __builtin_amdgcn_readfirstlane(sctx[b]);
    const int64_t pos = (int64_t)ctx + (row - row0);
    const int off = a.offsets ? a.offsets[b] : 0;
    if (row < row0 || ctx < 0 || off < 0 || pos + off >= a.max_position) continue;
    // requested ahead of their use: the page and the angles
    const int64_t slot = pos >> a.page_log2;
    const uint32_t id = slot < a.ld_table ? (uint32_t)a.table[(int64_t)b * a.ld_table + slot]
                                          : 0xffffffffu;
    f32x4 co[2] = {}, si[2] = {};             // pairs of the lane's dims: 8, or 4 interleaved
    if (a.rot) {
      const float* cs = a.cos_sin + (pos + off) * a.rot;
      const int at = !in_rot ? 0 : a.interleaved ? 4 * c : 8 * c - (second ? half : 0);
      const int more = a.interleaved ? 0 : 4;
      co[0] = load_any<f32x4>(cs + at);
      co[1] = load_any<f32x4>(cs + at + more);
      si[0] = load_any<f32x4>(cs + half + at);
      si[1] = load_any<f32x4>(cs + half + at + more);
    }
    const T* qrow = (const T*)a.q + (int64_t)row * a.ld_q;
    const T* krow = (const T*)a.k + (int64_t)row * a.ld_k;
    const T* vrow = (const T*)a.v + (int64_t)row * a.ld_v;
    const int g0 = slice * a.slice_groups;
    const int g1 = min(g0 + a.slice_groups, (per_row + HPW - 1) / HPW);
    T next[8];
    ask_head<D, T>(next, qrow, krow, vrow, g0 * HPW + lane / LPH, c, a.heads, a.kv_heads);
    for (int g = g0; g < g1; ++g) {
    T raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = next[i];
    ask_head<D, T>(next, qrow, krow, vrow, min(g + 1, g1 - 1) * HPW + lane / LPH, c, a.heads,
                   a.kv_heads);
    const int hh = g * HPW + lane / LPH;
    const bool live = hh < per_row;
    const bool is_q = hh < a.heads;
    const bool is_k = !is_q && hh < a.heads + a.kv_heads;
    const int kh = is_q ? 0 : is_k ? hh - a.heads : hh - a.heads - a.kv_heads;
    const bool turn = in_rot;

    float y[8];
    if (!is_q && !is_k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = (float)raw[i];         // V goes in as it is
    } else {
      double x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = (double)(float)raw[i];
      if (is_q ? a.qw != nullptr : a.kw != nullptr) {
        double ss = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fma(x[i], x[i], ss);
        ss += dpp_f64<DPP_XOR1>(ss);
        ss += dpp_f64<DPP_XOR2>(ss);
        ss += dpp_f64<DPP_MIRROR8>(ss);
        if constexpr (LPH >= 16) ss += dpp_f64<DPP_MIRROR16>(ss);
        if constexpr (LPH >= 32) ss += shfl_xor_f64(ss, 16);
        const double inv = rsqrt_f64(ss * (1.0 / D) + (double)a.eps);
        const double* w = sw[is_q ? 0 : 1] + 8 * c;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * (inv * w[i]);
      }
      if (a.rot) {
        if (a.interleaved) {
          if (turn) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const double u = x[2 * i], v = x[2 * i + 1];
              x[2 * i] = __builtin_fma(v, -(double)si[0][i], u * (double)co[0][i]);
              x[2 * i + 1] = __builtin_fma(u, (double)si[0][i], v * (double)co[0][i]);
            }
          }
        } else {
          // dim i of the first half turns with dim i + half: half/8 lanes away
          double y2[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y2[i] = shfl_f64(x[i], partner);
          if (turn) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              x[i] = __builtin_fma(y2[i], (double)(second ? si[i / 4][i % 4] : -si[i / 4][i % 4]),
                                   x[i] * (double)co[i / 4][i % 4]);
          }
        }
      }
      if (is_q) {
        if (live) {
          T r[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) r[i] = round_to<T>(x[i]);
          __builtin_memcpy((T*)a.q_out + (int64_t)row * a.ld_qout + (int64_t)hh * D + 8 * c, r,
                           sizeof(r));
        }
        continue;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = odd_f32(x[i]);
    }

    // the block of 32 dims (four lanes): smallest power of two that holds its largest
    // magnitude as 6 (codes end at 6), within [2^-126, 2^125]; 255 if one is not finite
    float amax = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      amax = __builtin_fmaxf(amax, __builtin_fabsf(y[i]));
      bad |= !(__builtin_fabsf(y[i]) < __builtin_inff());
    }
    amax = bad ? __builtin_inff() : amax;
    amax = __builtin_fmaxf(amax, dpp_f32<DPP_XOR1>(amax));
    amax = __builtin_fmaxf(amax, dpp_f32<DPP_XOR2>(amax));
    bad = amax == __builtin_inff();
    // amax = f 2^e, f in [1, 2): f <= 1.5 fits 6 * 2^(e-2), else 6 * 2^(e-1)
    const int e = __builtin_amdgcn_frexp_expf(amax) - 1;
    const float f = __builtin_amdgcn_ldexpf(amax, -e);
    int byte = e + 127 - (f > 1.5f ? 1 : 2);
    byte = amax > 0.f ? min(max(byte, 1), 252) : 1;
    // scaling by a power of two is exact down to where fp32 underflows, far below the
    // first border (only the sign is kept there); past the largest code it saturates
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float z = __builtin_amdgcn_ldexpf(y[i], 127 - byte);
      z = y[i] < 0.f ? __builtin_fminf(z, -1e-30f) : z + 0.f;
      y[i] = bad ? 0.f : z;
    }
    const uint32_t word = pack_codes(y);                      // the lane's 8 codes
    if (bad) byte = 255;
    if (!live) continue;

    if (a.k_val) {                            // the values the cache now stands for
      const float sc = bad ? __builtin_nanf("") : __builtin_bit_cast(float, (uint32_t)byte << 23);
      const f32x2 y0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.f, 0);
      const f32x2 y1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.f, 1);
      const f32x2 y2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.f, 2);
      const f32x2 y3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.f, 3);
      const T r[8] = {(T)(y0[0] * sc), (T)(y0[1] * sc), (T)(y1[0] * sc), (T)(y1[1] * sc),
                      (T)(y2[0] * sc), (T)(y2[1] * sc), (T)(y3[0] * sc), (T)(y3[1] * sc)};
      T* dst = (T*)(is_k ? a.k_val : a.v_val) + ((int64_t)row * a.kv_heads + kh) * D + 8 * c;
      __builtin_memcpy(dst, r, sizeof(r));
    }
    if (id >= (uint64_t)a.num_pages) continue;
    const int P = a.page, t = (int)pos & (P - 1);
    uint8_t* u = a.pages + ((int64_t)id * a.kv_heads + kh) * unit_bytes(P, D);
    uint8_t* sc = u + (is_k ? off_ks(P, D) : off_vs(P, D)) + (t >> 3) * (D / 4) + (t & 7);
    if ((c & 3) == 0) sc[(c >> 2) * 8] = (uint8_t)byte;
    if (is_k) {
      *(uint32_t*)(u + t * (D / 2) + 4 * c) = word;
    } else {
      uint8_t* d = u + off_v(P, D) + (t >> 3) * (4 * D) + (t & 7) * (D / 32);
      if constexpr (D == 64) {                // two 16ths of the dims per lane
        *(uint16_t*)(d + (2 * c) * 16) = (uint16_t)word;
        *(uint16_t*)(d + (2 * c + 1) * 16) = (uint16_t)(word >> 16);
      } else if constexpr (D == 128) {
        *(uint32_t*)(d + c * 32) = word;
      } else {                                // half a 16th per lane
        *(uint32_t*)(d + (c >> 1) * 64 + (c & 1) * 4) = word;
      }
    }
    }
  }
}

// -------------------------------------------------------------------- pages

constexpr int MAX_PAGES = 1 << 24;
constexpr int CHUNK = 4096;                   // counts a workgroup looks at

// Sums over a workgroup of NT threads: inclusive in thread order, and the total.
template <int NT, typename I>
__device__ __forceinline__ I block_scan(I x, I* wsum, I& total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const I y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  if (lane == 63) wsum[w] = x;
  __syncthreads();
  I carry = 0;
  total = 0;
  for (int i = 0; i < NT / 64; ++i) {
    if (i < w) carry += wsum[i];
    total += wsum[i];
  }
  __syncthreads();
  return x + carry;
}

// The pages in use among a wave's 1,024 of a chunk: 64 at a time, a page per lane.
__device__ __forceinline__ void used_masks(const int32_t* refs, int num_pages, int w0,
                                           uint64_t (&mask)[16]) {
  const int lane = threadIdx.x & 63;
  int32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = refs[min(w0 + 64 * i + lane, num_pages - 1)];
#pragma unroll
  for (int i = 0; i < 16; ++i) mask[i] = __ballot(w0 + 64 * i + lane < num_pages && r[i] != 0);
}
__device__ __forceinline__ int wave_pages() {
  return blockIdx.x * CHUNK + (threadIdx.x >> 6) * (CHUNK / 4);
}

// Pages in use in each chunk of the pool.
__global__ __launch_bounds__(256) void k_count(const int32_t* __restrict__ refs, int num_pages,
                                               int32_t* __restrict__ used) {
  __shared__ int wsum[4];
  uint64_t mask[16];
  used_masks(refs, num_pages, wave_pages(), mask);
  int n = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) n += __builtin_popcountll(mask[i]);
  if ((threadIdx.x & 63) == 0) wsum[threadIdx.x >> 6] = n;
  __syncthreads();
  if (threadIdx.x == 0) used[blockIdx.x] = wsum[0] + wsum[1] + wsum[2] + wsum[3];
}

// Sum of used[0 .. upto) by a workgroup of 256, and of all of it.
__device__ __forceinline__ void used_before(const int32_t* used, int chunks, int upto, int* wsum,
                                            int& before, int& all) {
  int x = 0, y = 0;
  for (int i = threadIdx.x; i < chunks; i += 256) {
    const int u = used[i];
    y += u;
    if (i < upto) x += u;
  }
  block_scan<256, int>(x, wsum, before);
  block_scan<256, int>(y, wsum, all);
}

struct PageArgs {
  const int32_t* cu;
  int batch, page_log2;
  int32_t *seq_lens, *table;
  int64_t ld_table;
  int32_t* refs;
  int num_pages, chunks;
  uint8_t* pages;
  int64_t page_bytes, layer_bytes;
  int layers;
  int32_t *ctx, *status;
  // workspace
  int32_t* used;          // [chunks]
  uint64_t* bits;         // [words], in its place for small pools: a free page each
  int32_t* rank;          // [words] free pages before a word
  int32_t* dst;           // [batch] the page for a copy (small pools)
  int32_t* first;         // [batch + 1] rank of a request's first new page among the free ones
  int32_t* copy;          // [batch] page to copy into the request's first new page, or -1
  int copy_layers;        // workgroups that share a small pool's copies of one request
};

__device__ __forceinline__ int pages_of(int64_t n, int page_log2) {
  return (int)((n + (1 << page_log2) - 1) >> page_log2);
}

// What a request needs (a thread per request): its status without regard to the
// others, its new pages and the shared last page among them.
struct Need {
  int st, len, rows, tail, pages;
};
__device__ __forceinline__ Need need_of(const PageArgs& a) {
  const int b = threadIdx.x;
  Need n = {SV_ROW_BAD_K, 0, 0, -1, 0};
  if (b >= a.batch) return n;
  const int c0 = a.cu[b], c1 = a.cu[b + 1];
  n.len = a.seq_lens[b];
  if (c0 < 0 || c1 <= c0) return n;
  n.rows = c1 - c0;
  if (n.len < 0) {
    n.st = SV_ROW_BAD_PARAM;
    return n;
  }
  const int64_t want = ((int64_t)n.len + n.rows + (1 << a.page_log2) - 1) >> a.page_log2;
  const int have = pages_of(n.len, a.page_log2);
  if (want > a.ld_table) {
    n.st = SV_ROW_NO_PAGES;
    return n;
  }
  n.st = SV_ROW_OK;
  n.pages = (int)want - have;
  if (n.len & ((1 << a.page_log2) - 1)) {
    const int32_t id = a.table[(int64_t)b * a.ld_table + have - 1];
    if ((uint32_t)id >= (uint32_t)a.num_pages) {
      n.st = SV_ROW_BAD_PAGE;
      n.pages = 0;
    } else if (a.refs[id] > 1) {
      n.tail = id;
      n.pages += 1;
    }
  }
  return n;
}

// Ranks of the free pages for every request, in request order, by a workgroup of
// 1,024.  first, ctx, copy: in LDS, for the caller.
__device__ __forceinline__ void plan_requests(const PageArgs& a, Need n, int64_t free_pages,
                                              int64_t* wsum, int* first, int* ctx, int* copy) {
  const int b = threadIdx.x;
  // the first request whose offsets break the packing rule, and all behind it
  if (b == 0) first[MAX_BATCH] = a.batch;
  __syncthreads();
  if (b < a.batch && (a.cu[b] < 0 || a.cu[b + 1] < a.cu[b])) atomicMin(&first[MAX_BATCH], b);
  __syncthreads();
  if (b >= first[MAX_BATCH]) n = {SV_ROW_BAD_K, 0, 0, -1, 0};
  int64_t total;
  const int64_t need = n.pages, end = block_scan<1024, int64_t>(need, wsum, total);
  if (b < a.batch) {
    if (n.st == SV_ROW_OK && need > 0 && end > free_pages) n.st = SV_ROW_NO_PAGES;
    // (ranks past the pool are never handed out)
    first[b] = (int)min(end - need, (int64_t)MAX_PAGES);
    if (b == a.batch - 1) first[a.batch] = (int)min(end, (int64_t)MAX_PAGES);
    copy[b] = n.st == SV_ROW_OK ? n.tail : -1;
    ctx[b] = n.st == SV_ROW_OK ? n.len : -1;
    a.copy[b] = copy[b];
    a.ctx[b] = ctx[b];
    a.status[b] = n.st;
    if (n.st == SV_ROW_OK) a.seq_lens[b] = n.len + n.rows;
  }
}

__global__ __launch_bounds__(1024) void k_reserve_plan(PageArgs a) {
  __shared__ int64_t wsum[16];
  __shared__ int first[MAX_BATCH + 1], ctx[MAX_BATCH], copy[MAX_BATCH];
  int64_t free_pages = 0, all;
  for (int i = threadIdx.x; i < a.chunks; i += 1024) free_pages -= a.used[i];
  block_scan<1024, int64_t>(free_pages, wsum, all);
  plan_requests(a, need_of(a), all + a.num_pages, wsum, first, ctx, copy);
  __syncthreads();
  for (int i = threadIdx.x; i <= a.batch; i += 1024) a.first[i] = first[i];
}

// Free page p has rank `rank` among the free ones: it goes to the request whose
// range first[b] .. first[b+1] holds the rank (first, ctx and copy in LDS; ctx -1:
// the request failed, its pages stay free; copy >= 0: its first new page replaces
// the last it has).
__device__ __forceinline__ void give_page(const PageArgs& a, int p, int rank, const int* first,
                                          const int* ctx, const int* copy) {
  int lo = 0, hi = a.batch;                   // (ranges can be empty: the last start <= rank)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= rank) lo = mid;
    else hi = mid;
  }
  const int len = ctx[lo];
  if (len < 0) return;
  const int slot = pages_of(len, a.page_log2) - (copy[lo] >= 0) + rank - first[lo];
  a.table[(int64_t)lo * a.ld_table + slot] = p;
  a.refs[p] = 1;
}

// Hands out the free pages of a chunk by their rank.
__global__ __launch_bounds__(256) void k_reserve_assign(PageArgs a) {
  __shared__ int wsum[4];
  __shared__ int first[MAX_BATCH + 1], ctx[MAX_BATCH], copy[MAX_BATCH];
  int before, all;
  used_before(a.used, a.chunks, blockIdx.x, wsum, before, all);
  const int rank0 = (int)blockIdx.x * CHUNK - before;
  if (rank0 >= a.first[a.batch]) return;
  for (int i = threadIdx.x; i <= a.batch; i += 256) first[i] = a.first[i];
  for (int i = threadIdx.x; i < a.batch; i += 256) {
    ctx[i] = a.ctx[i];
    copy[i] = a.copy[i];
  }
  const int lane = threadIdx.x & 63, w0 = wave_pages();
  uint64_t mask[16];
  used_masks(a.refs, a.num_pages, w0, mask);
  int n = 0, total;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int in_pool = min(max(a.num_pages - (w0 + 64 * i), 0), 64);     // the others are free
    mask[i] = ~mask[i] & (in_pool == 64 ? ~0ull : (1ull << in_pool) - 1);
    n += __builtin_popcountll(mask[i]);
  }
  int rank = rank0 + (block_scan<256, int>(lane == 0 ? n : 0, wsum, total) - n);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int mine = rank + __builtin_popcountll(mask[i] & ((1ull << lane) - 1));
    if ((mask[i] >> lane & 1) && mine < first[a.batch])
      give_page(a, w0 + 64 * i + lane, mine, first, ctx, copy);
    rank += __builtin_popcountll(mask[i]);
  }
}

// Free bits of a pool, 64 pages per word, a wave per 4 words.
__global__ __launch_bounds__(256) void k_pool_bits(const int32_t* __restrict__ refs, int num_pages,
                                                   uint64_t* __restrict__ bits) {
  const int lane = threadIdx.x & 63;
  const int w0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = 64 * (w0 + i) + lane;
    const uint64_t m = __ballot(refs[min(p, num_pages - 1)] == 0 && p < num_pages);
    if (lane == 0) bits[w0 + i] = m;
  }
}

// Pools of at most 65,536 pages: the plan by one workgroup over the pool's free
// bits (the counts themselves are 256 KB, which one workgroup takes 20 us to read).
// It hands out itself what up to 64 words hold (a verify step; four words per wave)
// and leaves more (prompts) to the next launch.  It says also which page each shared
// tail goes to, so that copies and assignment are that one launch.  In a captured
// graph, with release: a step of 512 requests 18.8 us (20.0 with all of it left
// over), 64 requests that take 16,000 pages 19.0 us (27.8 with none).
constexpr int SMALL_POOL = 65536;
// The free pages of word w, by a wave.
__device__ __forceinline__ void hand_out(const PageArgs& a, int w, uint64_t bits, int rank,
                                         const int* first, const int* ctx, const int* copy) {
  const int lane = threadIdx.x & 63;
  const int r = rank + __builtin_popcountll(bits & ((1ull << lane) - 1));
  if ((bits >> lane & 1) && r < first[a.batch]) give_page(a, 64 * w + lane, r, first, ctx, copy);
}
__global__ __launch_bounds__(1024) void k_reserve_small(PageArgs a) {
  __shared__ int64_t wsum[16];
  __shared__ uint64_t bits[SMALL_POOL / 64];
  __shared__ int rank[SMALL_POOL / 64];
  __shared__ int first[MAX_BATCH + 1], ctx[MAX_BATCH], copy[MAX_BATCH];
  const int tid = threadIdx.x;
  const int words = (a.num_pages + 1023) / 1024 * 16;
  const uint64_t mine = tid < words ? a.bits[tid] : 0;
  const Need need = need_of(a);
  bits[tid] = mine;
  const int n = __builtin_popcountll(mine);
  int64_t free_pages;
  rank[tid] = (int)block_scan<1024, int64_t>(n, wsum, free_pages) - n;
  plan_requests(a, need, free_pages, wsum, first, ctx, copy);
  __syncthreads();
  const int want = first[a.batch];
  const int todo = __syncthreads_count(tid < words && rank[tid] < want);
  if (tid < words) a.rank[tid] = todo <= 64 ? 0x7fffffff : rank[tid];
  if (todo <= 64)
    for (int w = tid >> 6; w < todo; w += 16) hand_out(a, w, bits[w], rank[w], first, ctx, copy);
  for (int i = tid; i <= a.batch; i += 1024) a.first[i] = first[i];
  if (tid < a.batch && copy[tid] >= 0) {      // (such a request got its pages)
    int lo = 0, hi = words;                   // the last word with rank <= first[tid]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (rank[mid] <= first[tid]) lo = mid;
      else hi = mid;
    }
    int left = first[tid] - rank[lo], at = 0;
#pragma unroll
    for (int w = 32; w > 0; w >>= 1) {
      const int c = __builtin_popcountll(bits[lo] >> at & ((1ull << w) - 1));
      if (left >= c) {
        left -= c;
        at += w;
      }
    }
    a.dst[tid] = 64 * lo + at;
  }
}

// Copies a shared tail to its own page in one layer; the old page's count goes down.
__device__ __forceinline__ void copy_tail(const PageArgs& a, int src, int dst, int layer) {
  const u32x4* s = (const u32x4*)(a.pages + layer * a.layer_bytes + src * a.page_bytes);
  u32x4* d = (u32x4*)(a.pages + layer * a.layer_bytes + dst * a.page_bytes);
  for (int64_t i = threadIdx.x; i < a.page_bytes / 16; i += 256) d[i] = s[i];
  if (layer == 0 && threadIdx.x == 0) atomicSub(&a.refs[src], 1);
}

// The copies of all layers (first: they are the longest), then 1,024 pages per
// workgroup to hand out.  A workgroup per request and layer up to 1,024 layers, so that
// the grid stays under the 2^24 workgroups of 256 that a launch can have.
constexpr int MAX_COPY_LAYERS = 1024;
__global__ __launch_bounds__(256) void k_reserve_finish(PageArgs a) {
  if ((int)blockIdx.x < a.batch * a.copy_layers) {
    const int b = (int)blockIdx.x % a.batch, src = a.copy[b];
    if (src < 0) return;
    for (int layer = (int)blockIdx.x / a.batch; layer < a.layers; layer += a.copy_layers)
      copy_tail(a, src, a.dst[b], layer);
    return;
  }
  __shared__ int first[MAX_BATCH + 1], ctx[MAX_BATCH], copy[MAX_BATCH];
  const int w0 = ((int)blockIdx.x - a.batch * a.copy_layers) * 16;
  if (a.rank[w0] >= a.first[a.batch]) return;
  for (int i = threadIdx.x; i <= a.batch; i += 256) first[i] = a.first[i];
  for (int i = threadIdx.x; i < a.batch; i += 256) {
    ctx[i] = a.ctx[i];
    copy[i] = a.copy[i];
  }
  const int w = w0 + (threadIdx.x >> 6) * 4;
  uint64_t m[4];
  int rank[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = a.bits[w + i];
    rank[i] = a.rank[w + i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) hand_out(a, w + i, m[i], rank[i], first, ctx, copy);
}

// Larger pools: copies the shared tails once the pages are handed out.
__global__ __launch_bounds__(256) void k_copy_tails(PageArgs a) {
  const int b = blockIdx.x, src = a.copy[b];
  if (src < 0) return;
  const int dst = a.table[(int64_t)b * a.ld_table + pages_of(a.ctx[b], a.page_log2) - 1];
  copy_tail(a, src, dst, blockIdx.y);
}

// A workgroup per request; 512 of them take 3.7 us, a launch's latency.
__global__ __launch_bounds__(256) void k_release(const int32_t* __restrict__ give,
                                                 const int32_t* __restrict__ ctx, int page_log2,
                                                 int32_t* __restrict__ seq_lens,
                                                 int32_t* __restrict__ table, int64_t ld_table,
                                                 int32_t* __restrict__ refs, int num_pages,
                                                 int32_t* __restrict__ status) {
  const int b = blockIdx.x;
  const int len = seq_lens[b], g = give[b];
  const bool skip = ctx && ctx[b] < 0;
  __syncthreads();
  const int have = len < 0 ? 0 : pages_of(len, page_log2);
  int st = SV_ROW_OK;
  if (!skip && (len < 0 || g < 0 || g > len || have > ld_table)) st = SV_ROW_BAD_PARAM;
  bool bad = false;
  if (!skip && st == SV_ROW_OK) {
    int32_t* row = table + (int64_t)b * ld_table;
    for (int s = pages_of(len - g, page_log2) + threadIdx.x; s < have; s += 256) {
      const int32_t id = row[s];
      if ((uint32_t)id < (uint32_t)num_pages) atomicSub(&refs[id], 1);
      else bad = true;
      row[s] = -1;
    }
  }
  const bool any_bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    status[b] = any_bad ? SV_ROW_BAD_PAGE : st;
    if (!skip && st == SV_ROW_OK) seq_lens[b] = len - g;
  }
}

// One workgroup per pair: its status, and with COPY (few pairs, one launch) the
// fork itself.  What a pair decides does not depend on what another has written: it
// reads the length of its src, which is nobody's dst, and of its dst, which no
// earlier pair names.
template <bool COPY>
__global__ __launch_bounds__(256) void k_fork_check(const int32_t* __restrict__ src,
                                                    const int32_t* __restrict__ dst,
                                                    const int32_t* __restrict__ lens, int pairs,
                                                    int seqs, int page_log2, int32_t* seq_lens,
                                                    int32_t* table, int64_t ld_table, int32_t* refs,
                                                    int num_pages, int32_t* __restrict__ status) {
  const int i = blockIdx.x, s = src[i], d = dst[i];
  bool clash = false;       // an earlier pair writes d, or some pair writes s
  for (int k = threadIdx.x; k < pairs; k += 256) {
    const int t = dst[k];
    clash |= (k < i && t == d) || t == s;
  }
  int st = SV_ROW_OK, n = 0, held = 0;
  if (__syncthreads_or(clash) || (uint32_t)s >= (uint32_t)seqs || (uint32_t)d >= (uint32_t)seqs)
    st = SV_ROW_BAD_PARAM;
  const int32_t* from = table + (int64_t)(st == SV_ROW_OK ? s : 0) * ld_table;
  if (st == SV_ROW_OK) {
    const int have = seq_lens[s];
    n = lens ? lens[i] : have;
    if (seq_lens[d] != 0 || n < 0 || n > have) st = SV_ROW_BAD_PARAM;
    else {
      held = pages_of(n, page_log2);
      bool bad = held > ld_table;
      if (!bad)
        for (int k = threadIdx.x; k < held; k += 256)
          bad |= (uint32_t)from[k] >= (uint32_t)num_pages;
      if (__syncthreads_or(bad)) st = SV_ROW_BAD_PAGE;
    }
  }
  if (COPY && st == SV_ROW_OK)
    for (int k = threadIdx.x; k < held; k += 256) {
      const int32_t id = from[k];
      table[(int64_t)d * ld_table + k] = id;
      atomicAdd(&refs[id], 1);
    }
  __syncthreads();          // (every thread has read the length of d)
  if (threadIdx.x == 0) {
    status[i] = st;
    if (COPY && st == SV_ROW_OK) seq_lens[d] = n;
  }
}

// Workgroup (i, j): where pair i is the first good one of its src, every gridDim.y-th
// 256 entries of that row go to every good dst of the src, and each page's count goes up once
// by how many took it.  Device-wide atomics are what bounds a fork: 896 pairs of 128
// prompts take 8 us here after 5 for their statuses, and 18 with a count per page and
// pair in the one-launch form.
__global__ __launch_bounds__(256) void k_fork_copy(const int32_t* __restrict__ src,
                                                   const int32_t* __restrict__ dst,
                                                   const int32_t* __restrict__ lens, int pairs,
                                                   int page_log2, int32_t* seq_lens, int32_t* table,
                                                   int64_t ld_table, int32_t* refs,
                                                   const int32_t* __restrict__ status) {
  __shared__ int to[MAX_BATCH], held[MAX_BATCH], count;
  const int i = blockIdx.x;
  if (status[i] != SV_ROW_OK) return;
  const int s = src[i];
  if (threadIdx.x == 0) count = 0;
  __syncthreads();
  bool later = false;
  const int have = seq_lens[s];               // (a src is nobody's dst)
  for (int k = threadIdx.x; k < pairs; k += 256)
    if (src[k] == s && status[k] == SV_ROW_OK) {
      later |= k < i;
      const int n = lens ? lens[k] : have, at = atomicAdd(&count, 1);
      to[at] = dst[k];
      held[at] = pages_of(n, page_log2);
      if (blockIdx.y == 0 && k >= i) seq_lens[dst[k]] = n;
    }
  if (__syncthreads_or(later)) return;
  // (a length past the table row is nobody's held pages: they were checked)
  const int pages = (int)min((int64_t)pages_of(have, page_log2), ld_table);
  for (int k = (int)blockIdx.y * 256 + threadIdx.x; k < pages; k += (int)gridDim.y * 256) {
    const int32_t id = table[(int64_t)s * ld_table + k];
    int took = 0;
    for (int m = 0; m < count; ++m)
      if (k < held[m]) {
        table[(int64_t)to[m] * ld_table + k] = id;
        ++took;
      }
    if (took) atomicAdd(&refs[id], took);
  }
}

struct CompactArgs {
  int seqs, page_log2;
  const int32_t* seq_lens;
  int32_t* table;
  int64_t ld_table;
  int32_t* refs;
  int num_pages, chunks;
  uint8_t* pages;
  int64_t page_bytes, layer_bytes;
  int layers;
  int32_t* live;
  int32_t* used;          // [chunks]
  int32_t* counts;        // [1] pages to move
  int32_t* hole;          // free pages below `live`, ascending
  int32_t* mover;         // pages in use from `live` on, descending
  int32_t* place;         // a mover's index in that order, by page
  int copy_blocks;
};

// With L pages in use: the free ids below L (holes) and the used ids from L on
// (movers) are equally many; the i-th mover from below goes to the i-th hole.
__global__ __launch_bounds__(256) void k_compact_rank(CompactArgs a) {
  __shared__ int wsum[4];
  int before, live;
  used_before(a.used, a.chunks, blockIdx.x, wsum, before, live);
  const int lane = threadIdx.x & 63, w0 = wave_pages();
  uint64_t mask[16];
  used_masks(a.refs, a.num_pages, w0, mask);
  int n = 0, total;
#pragma unroll
  for (int i = 0; i < 16; ++i) n += __builtin_popcountll(mask[i]);
  // used pages before the wave's
  int rank = before + block_scan<256, int>(lane == 0 ? n : 0, wsum, total) - n;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int p = w0 + 64 * i + lane;
    const int r = rank + __builtin_popcountll(mask[i] & ((1ull << lane) - 1));
    const bool used = mask[i] >> lane & 1;
    if (p < a.num_pages) {
      if (p == live) a.counts[0] = live - r;
      if (p < live && !used) a.hole[p - r] = p;
      if (p >= live && used) {
        a.mover[live - 1 - r] = p;
        a.place[p] = live - 1 - r;
      }
    }
    rank += __builtin_popcountll(mask[i]);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.live[0] = live;
    if (live == a.num_pages) a.counts[0] = 0;
  }
}

// 16 KB per workgroup and turn, four vectors per thread on their way at once: 227 MB
// read and written in 99 us (4.6 TB/s; a plain copy of 1 GiB reaches 5.1), after 10 us
// for counts and ranks.
__global__ __launch_bounds__(256) void k_compact_move(CompactArgs a) {
  const int moves = a.counts[0], live = a.live[0];
  if ((int)blockIdx.x >= a.copy_blocks) {     // a sequence's table
    const int b = (int)blockIdx.x - a.copy_blocks;
    const int len = a.seq_lens[b];
    const int64_t held = len < 0 ? 0 : pages_of(len, a.page_log2);
    int32_t* row = a.table + (int64_t)b * a.ld_table;
    for (int64_t s = threadIdx.x; s < held && s < a.ld_table; s += 256) {
      const int32_t id = row[s];
      if (id >= live && id < a.num_pages) {
        // a page the counts call free (a table at odds with them) keeps its id
        const uint32_t at = (uint32_t)a.place[id];
        if (at < (uint32_t)moves && a.mover[at] == id) row[s] = a.hole[moves - 1 - at];
      }
    }
    return;
  }
  const int64_t vecs = a.page_bytes / 16;
  const int64_t segs = (vecs + 1023) / 1024;
  const int64_t units = (int64_t)moves * a.layers * segs;
  for (int64_t u = blockIdx.x; u < units; u += a.copy_blocks) {
    const int64_t seg = u % segs, rest = u / segs;
    const int layer = (int)(rest % a.layers), i = (int)(rest / a.layers);
    const int64_t from = a.mover[moves - 1 - i], to = a.hole[i];
    const u32x4* s = (const u32x4*)(a.pages + layer * a.layer_bytes + from * a.page_bytes);
    u32x4* d = (u32x4*)(a.pages + layer * a.layer_bytes + to * a.page_bytes);
    u32x4 x[4];
    const int64_t v0 = seg * 1024 + threadIdx.x;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (v0 + 256 * k < vecs) x[k] = s[v0 + 256 * k];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (v0 + 256 * k < vecs) d[v0 + 256 * k] = x[k];
    if (layer == 0 && seg == 0 && threadIdx.x == 0) {
      a.refs[to] = a.refs[from];
      a.refs[from] = 0;
    }
  }
}

// ---- host side

static size_t round16(size_t x) { return (x + 15) / 16 * 16; }
static int chunks_of(int64_t num_pages) { return (int)((num_pages + CHUNK - 1) / CHUNK); }

// Reserve's free bits and their ranks (small pools; whole workgroups of 16 words) or
// chunk counts.
static size_t head_bytes(int64_t num_pages) {
  return num_pages <= SMALL_POOL ? 192 * (size_t)((num_pages + 1023) / 1024)
                                 : round16(4 * (size_t)chunks_of(num_pages));
}

static bool pool_ok(int seqs, int page, int64_t ld_table, int64_t num_pages) {
  return seqs >= 1 && seqs <= MAX_BATCH && page_ok(page) && ld_table >= 1 &&
         ld_table <= (1 << 30) / page && num_pages >= 1 && num_pages <= MAX_PAGES;
}

template <int D, typename T>
static int launch_append(AppendArgs a, hipStream_t s) {
  // a row per wave where that fills the device (4 waves per SIMD), else slices of rows
  constexpr int HPW = 512 / D;
  const int groups = (a.heads + 2 * a.kv_heads + HPW - 1) / HPW;
  int slices = 4096 / a.total_rows + 1;
  if (slices > groups) slices = groups;
  a.slice_groups = (groups + slices - 1) / slices;
  a.slices = (groups + a.slice_groups - 1) / a.slice_groups;
  a.tasks = a.total_rows * a.slices;          // (the caller: below 2^31)
  const int most = sizeof(T) == 2 ? 1024 : D == 256 ? 512 : 768;   // what the device holds at once
  const int blocks = min((a.tasks + 3) / 4, most);
  a.data_blocks = blocks;
  hipLaunchKernelGGL((k_append<D, T>), dim3((unsigned)blocks + (a.batch + 3) / 4), dim3(256), 0, s, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_LAUNCH;
}

}  // namespace svk

using namespace svk;

extern "C" {

size_t spec_kv_page_bytes(int kv_heads, int head_dim, int page_size) {
  if (kv_heads < 1 || kv_heads > 1024 || !dim_ok(head_dim) || !page_ok(page_size)) return 0;
  return (size_t)(kv_heads * unit_bytes(page_size, head_dim));
}

int spec_kv_append_at(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                      int64_t ld_v, int dtype, const float* q_weight, const float* k_weight, float eps,
                      const float* cos_sin, int max_position, int rot_dim, int interleaved,
                      const int32_t* cu_seqlens, const int32_t* context_lens,
                      const int32_t* position_offsets, int batch, int total_rows, int heads,
                      int kv_heads, int head_dim, void* pages, int64_t num_pages, int page_size,
                      const int32_t* page_table, int64_t ld_table, void* q_out, int64_t ld_qout,
                      void* k_values, void* v_values, int32_t* status, void* stream) {
  if (!q || !k || !v || !cu_seqlens || !context_lens || !pages || !page_table || !q_out || !status ||
      (rot_dim != 0 && !cos_sin) || (!k_values) != (!v_values))
    return SV_ERR_NULL;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  const int64_t d = head_dim;
  if (!pool_ok(batch, page_size, ld_table, num_pages) || !dim_ok(head_dim) || total_rows < 1 ||
      kv_heads < 1 || heads < kv_heads || heads > 1024 || heads % kv_heads != 0 ||
      ld_q < heads * d || ld_k < kv_heads * d || ld_v < kv_heads * d || ld_qout < heads * d ||
      rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0 || (rot_dim && max_position < 1) ||
      !(eps >= 0.f) || !(eps <= 1.f) || !aligned16(pages) ||
      (int64_t)total_rows * (heads + 2 * kv_heads) >= (1ll << 31) - 65536)
    return SV_ERR_SHAPE;
  AppendArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.ld_q = ld_q;
  a.ld_k = ld_k;
  a.ld_v = ld_v;
  a.qw = q_weight;
  a.kw = k_weight;
  a.eps = eps;
  a.cos_sin = cos_sin;
  a.max_position = rot_dim ? max_position : 0x7fffffff;
  a.rot = rot_dim;
  a.interleaved = interleaved;
  a.cu = cu_seqlens;
  a.ctx = context_lens;
  a.offsets = position_offsets;
  a.batch = batch;
  a.total_rows = total_rows;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.pages = (uint8_t*)pages;
  a.num_pages = num_pages;
  a.page = page_size;
  a.page_log2 = __builtin_ctz((unsigned)page_size);
  a.table = page_table;
  a.ld_table = ld_table;
  a.q_out = q_out;
  a.ld_qout = ld_qout;
  a.k_val = k_values;
  a.v_val = v_values;
  a.status = status;
  a.data_blocks = 0;
  hipStream_t s = (hipStream_t)stream;
  if (dtype == SV_BF16)
    return head_dim == 64    ? launch_append<64, __bf16>(a, s)
           : head_dim == 128 ? launch_append<128, __bf16>(a, s)
                             : launch_append<256, __bf16>(a, s);
  return head_dim == 64    ? launch_append<64, float>(a, s)
         : head_dim == 128 ? launch_append<128, float>(a, s)
                           : launch_append<256, float>(a, s);
}

int spec_kv_append(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                   int64_t ld_v, int dtype, const float* q_weight, const float* k_weight, float eps,
                   const float* cos_sin, int max_position, int rot_dim, int interleaved,
                   const int32_t* cu_seqlens, const int32_t* context_lens, int batch,
                   int total_rows, int heads, int kv_heads, int head_dim, void* pages,
                   int64_t num_pages, int page_size, const int32_t* page_table, int64_t ld_table,
                   void* q_out, int64_t ld_qout, void* k_values, void* v_values, int32_t* status,
                   void* stream) {
  return spec_kv_append_at(q, ld_q, k, ld_k, v, ld_v, dtype, q_weight, k_weight, eps, cos_sin,
                           max_position, rot_dim, interleaved, cu_seqlens, context_lens, nullptr,
                           batch, total_rows, heads, kv_heads, head_dim, pages, num_pages,
                           page_size, page_table, ld_table, q_out, ld_qout, k_values, v_values,
                           status, stream);
}

size_t spec_kv_pages_workspace_bytes(int seqs, int64_t num_pages) {
  if (!pool_ok(seqs, 16, 1, num_pages)) return 0;
  // reserve: used, first, copy, dst; compact: used, one count, three words per page
  const size_t used = round16(4 * (size_t)chunks_of(num_pages));
  const size_t reserve = head_bytes(num_pages) + round16(4 * ((size_t)seqs + 1)) + 2 * round16(4 * (size_t)seqs);
  const size_t compact = used + 16 + 3 * round16(4 * (size_t)num_pages);
  return reserve > compact ? reserve : compact;
}

int spec_kv_reserve(const int32_t* cu_seqlens, int batch, int page_size, int32_t* seq_lens,
                    int32_t* page_table, int64_t ld_table, int32_t* ref_counts, int64_t num_pages,
                    void* pages, int64_t page_bytes, int layers, int64_t layer_bytes,
                    int32_t* context_lens, int32_t* status, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!cu_seqlens || !seq_lens || !page_table || !ref_counts || !pages || !context_lens || !status ||
      !workspace)
    return SV_ERR_NULL;
  if (!pool_ok(batch, page_size, ld_table, num_pages) || page_bytes < 16 || page_bytes % 16 != 0 ||
      layers < 1 || layers > 65535 ||
      (layers > 1 && (layer_bytes % 16 != 0 || layer_bytes < num_pages * page_bytes)) || !aligned16(pages) ||
      !aligned16(workspace))
    return SV_ERR_SHAPE;
  if (workspace_bytes < spec_kv_pages_workspace_bytes(batch, num_pages)) return SV_ERR_WORKSPACE;
  PageArgs a;
  a.cu = cu_seqlens;
  a.batch = batch;
  a.page_log2 = __builtin_ctz((unsigned)page_size);
  a.seq_lens = seq_lens;
  a.table = page_table;
  a.ld_table = ld_table;
  a.refs = ref_counts;
  a.num_pages = (int)num_pages;
  a.chunks = chunks_of(num_pages);
  a.pages = (uint8_t*)pages;
  a.page_bytes = page_bytes;
  a.layer_bytes = layer_bytes;
  a.layers = layers;
  a.copy_layers = layers < MAX_COPY_LAYERS ? layers : MAX_COPY_LAYERS;
  a.ctx = context_lens;
  a.status = status;
  uint8_t* w = (uint8_t*)workspace;
  a.used = (int32_t*)w;
  a.bits = (uint64_t*)w;
  a.rank = (int32_t*)(w + 128 * (size_t)((num_pages + 1023) / 1024));
  w += head_bytes(num_pages);
  a.first = (int32_t*)w;
  w += round16(4 * ((size_t)batch + 1));
  a.copy = (int32_t*)w;
  a.dst = (int32_t*)(w + round16(4 * (size_t)batch));
  hipStream_t s = (hipStream_t)stream;
  if (a.num_pages <= SMALL_POOL) {
    const int groups = (a.num_pages + 1023) / 1024;
    hipLaunchKernelGGL(k_pool_bits, dim3(groups), dim3(256), 0, s, a.refs, a.num_pages, a.bits);
    hipLaunchKernelGGL(k_reserve_small, dim3(1), dim3(1024), 0, s, a);
    hipLaunchKernelGGL(k_reserve_finish, dim3(batch * a.copy_layers + groups), dim3(256), 0, s, a);
  } else {
    hipLaunchKernelGGL(k_count, dim3(a.chunks), dim3(256), 0, s, a.refs, a.num_pages, a.used);
    hipLaunchKernelGGL(k_reserve_plan, dim3(1), dim3(1024), 0, s, a);
    hipLaunchKernelGGL(k_reserve_assign, dim3(a.chunks), dim3(256), 0, s, a);
    hipLaunchKernelGGL(k_copy_tails, dim3(batch, layers), dim3(256), 0, s, a);
  }
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_LAUNCH;
}

int spec_kv_release(const int32_t* rollback, const int32_t* context_lens, int batch, int page_size,
                    int32_t* seq_lens, int32_t* page_table, int64_t ld_table, int32_t* ref_counts,
                    int64_t num_pages, int32_t* status, void* stream) {
  if (!rollback || !seq_lens || !page_table || !ref_counts || !status) return SV_ERR_NULL;
  if (!pool_ok(batch, page_size, ld_table, num_pages)) return SV_ERR_SHAPE;
  hipLaunchKernelGGL(k_release, dim3(batch), dim3(256), 0, (hipStream_t)stream, rollback,
                     context_lens, __builtin_ctz((unsigned)page_size), seq_lens, page_table,
                     ld_table, ref_counts, (int)num_pages, status);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_LAUNCH;
}

int spec_kv_fork(const int32_t* src, const int32_t* dst, const int32_t* lens, int pairs, int seqs,
                 int page_size, int32_t* seq_lens, int32_t* page_table, int64_t ld_table,
                 int32_t* ref_counts, int64_t num_pages, int32_t* status, void* stream) {
  if (!src || !dst || !seq_lens || !page_table || !ref_counts || !status) return SV_ERR_NULL;
  if (!pool_ok(seqs, page_size, ld_table, num_pages) || pairs < 1 || pairs > MAX_BATCH)
    return SV_ERR_SHAPE;
  const int log2 = __builtin_ctz((unsigned)page_size);
  hipStream_t s = (hipStream_t)stream;
  // a launch less for few pairs (64 of 8 prompts: 11 us a call against 14), counts
  // grouped by src for many (896 of 128 prompts: 16 us against 21)
  if (pairs <= 128) {
    hipLaunchKernelGGL(k_fork_check<true>, dim3(pairs), dim3(256), 0, s, src, dst, lens, pairs, seqs,
                       log2, seq_lens, page_table, ld_table, ref_counts, (int)num_pages, status);
    return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_LAUNCH;
  }
  hipLaunchKernelGGL(k_fork_check<false>, dim3(pairs), dim3(256), 0, s, src, dst, lens, pairs, seqs,
                     log2, seq_lens, page_table, ld_table, ref_counts, (int)num_pages, status);
  const int64_t splits = (ld_table + 255) / 256;
  hipLaunchKernelGGL(k_fork_copy, dim3(pairs, (unsigned)(splits < 16 ? splits : 16)), dim3(256), 0, s,
                     src, dst, lens, pairs, log2, seq_lens, page_table, ld_table, ref_counts,
                     status);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_LAUNCH;
}

int spec_kv_compact(int seqs, int page_size, const int32_t* seq_lens, int32_t* page_table,
                    int64_t ld_table, int32_t* ref_counts, int64_t num_pages, void* pages,
                    int64_t page_bytes, int layers, int64_t layer_bytes, int32_t* live,
                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!seq_lens || !page_table || !ref_counts || !pages || !live || !workspace) return SV_ERR_NULL;
  if (!pool_ok(seqs, page_size, ld_table, num_pages) || page_bytes < 16 || page_bytes % 16 != 0 ||
      layers < 1 || layers > 65535 ||
      (layers > 1 && (layer_bytes % 16 != 0 || layer_bytes < num_pages * page_bytes)) || !aligned16(pages) ||
      !aligned16(workspace))
    return SV_ERR_SHAPE;
  if (workspace_bytes < spec_kv_pages_workspace_bytes(seqs, num_pages)) return SV_ERR_WORKSPACE;
  CompactArgs a;
  a.seqs = seqs;
  a.page_log2 = __builtin_ctz((unsigned)page_size);
  a.seq_lens = seq_lens;
  a.table = page_table;
  a.ld_table = ld_table;
  a.refs = ref_counts;
  a.num_pages = (int)num_pages;
  a.chunks = chunks_of(num_pages);
  a.pages = (uint8_t*)pages;
  a.page_bytes = page_bytes;
  a.layer_bytes = layer_bytes;
  a.layers = layers;
  a.live = live;
  uint8_t* w = (uint8_t*)workspace;
  a.used = (int32_t*)w;
  w += round16(4 * (size_t)a.chunks);
  a.counts = (int32_t*)w;
  w += 16;
  const size_t per = round16(4 * (size_t)num_pages);
  a.hole = (int32_t*)w;
  a.mover = (int32_t*)(w + per);
  a.place = (int32_t*)(w + 2 * per);
  a.copy_blocks = 2048;
  hipStream_t s = (hipStream_t)stream;
  hipLaunchKernelGGL(k_count, dim3(a.chunks), dim3(256), 0, s, a.refs, a.num_pages, a.used);
  hipLaunchKernelGGL(k_compact_rank, dim3(a.chunks), dim3(256), 0, s, a);
  hipLaunchKernelGGL(k_compact_move, dim3(a.copy_blocks + seqs), dim3(256), 0, s, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_LAUNCH;
}

}  // extern "C"
