// kvprompt.hip -- spec_kv_prompt_attention: attention of whole prompts, any number
// of rows per request, over the 4-bit paged cache (include/specverify_cache.h
// states the operator).
//
// For request b, row j (position c+j) and query head h over KV head h/G:
//   out = sum_t exp(scale q.k_t - m) v_t / sum_t exp(scale q.k_t - m)
// over the visible t, in one pass with a running maximum m and sum.
//
// Two launches: k_prompt_prepare lists the work and turns the cache of the call's requests
// into bf16 once, and k_prompt takes it from there (a third joins the parts of rows whose
// context was split).
//
// Widening once, not per workgroup: a tile of 32 tokens is used by every block of rows
// behind it, rows * G / 256 times.  The widened tile is laid out as the matrix
// instructions' operands, [instruction][lane][8 values], so that its way through LDS is
// straight copies and reads without bank conflicts.  It takes 29 us of the 1,850 for one prompt
// of 15,991 rows, 23 of 297 for four of 1,500 to 4,000, 65 of 251 for two of 150 to 600 after
// 8,000 to 30,000 positions.  Latency bounds it: 45 MB read and 164 written in those 65 us are
// 3.2 TB/s of the 5.1 that a copy reaches, with the vector units 18 % busy; a wave has two or
// three tiles, each a chain of table, codes and stores with nothing else on its way.
//
// k_prompt: a workgroup of 4 or 8 waves takes one KV head and 32 of the request's rows * G
// query rows for each wave (the G heads of a row side by side).  Per tile it computes
// S^T[token][row] = K Q^T, then O^T[dim][row] += V^T P^T with v_mfma_f32_32x32x16_bf16.  With
// tokens as the rows of S^T a lane holds scores of ONE query row, for 16 of the tile's tokens:
// statistics are per lane, and the weights are the next product's operand as they are (V is
// laid out in the order of tokens in which the accumulators hold them).
//
// Roundings: bf16 rows' weights are rounded to bf16 for the second product (and summed as
// rounded), as the matrix instruction takes them: results are 0.0017 to 0.0023 of their norm from
// 64 bits.  Two bf16 terms per weight would leave the result's own rounding (0.0015 to 0.0017), for
// 2,650 us instead of 1,850 for the prompt below and 86 instead of 79 for 64 short ones.  fp32
// rows' queries and weights go in as three bf16 terms, exactly.  Scores, statistics and sums are
// fp32.
//
// What bounds it: the waves' alternation of products and softmax, matrix instructions 52 % of
// the time, vector ones 38 % (one prompt of 15,991 rows, 32 heads over 8 of D=128: 1.13
// PFLOP/s, where a large bf16 matrix product reaches 1.20 to 1.27; four prompts of 1,500 to
// 4,000 rows 0.80, their last workgroups ending alone).  Within a wave nothing hides the loads of
// the next stage: the compiler takes either half of the buffer for what they write, and has
// them waited for before the stage's first product; other waves' products run meanwhile.  Tried
// with that wait, and slower: the next tile's scores ahead of this one's softmax (2,307 us against
// 2,220 of the same kernel without, for the first of these), a barrier per tile over a ring of
// buffers.

#include "kv_common.h"
#include "row_ranges.h"

namespace svk {
namespace prompt {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int TILE = 32;                     // tokens
constexpr float LOG2E = 1.44269504088896340736f;
// the running maximum is raised when a score passes it by this much in powers of two
// (weights stay below 2^8), and counted from its rounded product with the scale, held
// within +-FAR; past it weights become infinite, or all 0, and their row NaN
constexpr float RAISE = 8.0f;
constexpr float FAR = 1073741824.0f;         // 2^30

constexpr int tile_bytes(int d) { return TILE * d * 2 * 2; }    // K, then V, in bf16

// A workgroup's work: rows [rb * block_rows, ...) of request b's rows * G over a chunk of their
// context; with the request's numbers, so that one load tells a workgroup all (ctx < 0: its rows
// are NaN).
struct Item {
  int b, rb, chunk, block, row0, rows, ctx, tile;
};
// What the plan writes.
struct Head {
  int items, blocks;
};

struct Args {
  const void* q;
  int64_t ld_q;
  const int32_t* cu;
  const int32_t* ctx;
  int batch, total_rows, heads, kv_heads, group;
  const uint8_t* pages;
  int64_t num_pages;
  int page, page_log2, unit;
  const int32_t* table;
  int64_t ld_table;
  int max_context;
  int64_t total_context;
  float scale;
  int window, sinks;
  void* out;
  int64_t ld_out;
  int32_t* status;
  int block_rows, max_blocks, chunks, chunk_tiles;
  int64_t max_tiles;
  // workspace
  Head* head;
  Item* items;                               // by falling work
  Item* blocks;                              // chunk 0 of every block, in order
  uint8_t* wide;                             // [kv_heads][max_tiles][tile_bytes]
  // V blocks stored as NaN: [kv_heads][max_tiles] a tile's tokens that have some, and
  // [kv_heads][max_tiles][32] which ones
  uint32_t* odd;
  uint8_t* odd_blocks;
  float* part;
};

// Tiles that a request's rows see together: the first `early` of the sequence, then those
// from `tile0` on.
struct Span {
  int n, first, early, tile0, tiles;
};
__device__ __forceinline__ Span span_of(int ctx, int rows, int window, int sinks) {
  Span s;
  s.n = ctx + rows;
  s.first = window > 0 ? max(0, ctx - window + 1) : 0;
  s.tile0 = s.first / TILE;
  s.early = window > 0 ? min((sinks + TILE - 1) / TILE, s.tile0) : 0;
  s.tiles = s.early + (s.n - 1) / TILE - s.tile0 + 1;
  return s;
}
// The same of the rows first_row .. last_row alone.
__device__ __forceinline__ Span block_span(int ctx, int first_row, int last_row, int window, int sinks) {
  return span_of(ctx + first_row, last_row - first_row + 1, window, sinks);
}

// The requests of a call, in LDS: statuses by offsets and lengths alone, contexts (-1 where
// a request has none), and running counts of row blocks and widened tiles.
struct Requests {
  int red[4][4], status[MAX_BATCH], row0[MAX_BATCH], rows[MAX_BATCH], ctx[MAX_BATCH];
  int block[MAX_BATCH + 1], tile[MAX_BATCH + 1];
  long long held[4];
};
// 256 threads, four requests in a row each.
__device__ __forceinline__ void find_requests(const Args& a, Requests& q) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int c0[4], c1[4], cx[4], broken = a.batch;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = min(4 * tid + i, a.batch - 1);
    c0[i] = a.cu[b];
    c1[i] = a.cu[b + 1];
    cx[i] = a.ctx[b];
  }
#pragma unroll
  for (int i = 3; i >= 0; --i)
    if (4 * tid + i < a.batch && (c0[i] < 0 || c1[i] < c0[i] || c1[i] > a.total_rows)) broken = 4 * tid + i;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) broken = min(broken, __shfl_xor(broken, d));
  if (lane == 0) q.red[0][wave] = broken;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) broken = min(broken, q.red[0][w]);
  int st[4];
  long long held[4], sum = 0;                 // what the requests hold so far, against the call's bound
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rows = c1[i] - c0[i];
    st[i] = 4 * tid + i < broken && rows >= 1 ? SV_ROW_OK : SV_ROW_BAD_K;
    if (st[i] == SV_ROW_OK && (cx[i] < 0 || (int64_t)cx[i] + rows > a.max_context)) st[i] = SV_ROW_BAD_PARAM;
    if (st[i] == SV_ROW_OK) sum += (long long)cx[i] + rows;
    held[i] = sum;
  }
  long long upto = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const long long y = __shfl_up(upto, d);
    if (lane >= d) upto += y;
  }
  if (lane == 63) q.held[wave] = upto;
  __syncthreads();
  for (int w = 0; w < wave; ++w) upto += q.held[w];
  int nb[4], nt[4], sb = 0, stl = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (st[i] == SV_ROW_OK && upto - sum + held[i] > a.total_context) st[i] = SV_ROW_BAD_PARAM;
    const int rows = c1[i] - c0[i];
    const int64_t R = st[i] == SV_ROW_BAD_K ? 0 : (int64_t)rows * a.group;
    sb += nb[i] = (int)((R + a.block_rows - 1) / a.block_rows);
    stl += nt[i] = st[i] == SV_ROW_OK ? span_of(cx[i], rows, a.window, a.sinks).tiles : 0;
  }
  int ub = sb, ut = stl;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(ub, d), z = __shfl_up(ut, d);
    if (lane >= d) {
      ub += y;
      ut += z;
    }
  }
  if (lane == 63) {
    q.red[1][wave] = ub;
    q.red[2][wave] = ut;
  }
  __syncthreads();
  for (int w = 0; w < wave; ++w) {
    ub += q.red[1][w];
    ut += q.red[2][w];
  }
  ub -= sb;
  ut -= stl;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = 4 * tid + i;
    q.status[b] = st[i];
    q.row0[b] = c0[i];
    q.rows[b] = c1[i] - c0[i];
    q.ctx[b] = st[i] == SV_ROW_OK ? cx[i] : -1;
    q.block[b] = ub;
    q.tile[b] = ut;
    ub += nb[i];
    ut += nt[i];
  }
  if (tid == 255) {
    q.block[MAX_BATCH] = ub;
    q.tile[MAX_BATCH] = ut;
  }
  __syncthreads();
}
// The last request whose count is at most x.
__device__ __forceinline__ int request_at(const int* count, int batch, int x) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (count[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The 16 positions from t0 on: whether some row of the request sees one of them.
__device__ __forceinline__ bool half_needed(const Args& a, const Span& sp, int t0) {
  return t0 < sp.n && (t0 + 16 > sp.first || (a.window > 0 && t0 < min(a.sinks, sp.first)));
}
__device__ __forceinline__ int base_of(const Span& sp, int i) {
  return (i < sp.early ? i : i - sp.early + sp.tile0) * TILE;
}
// Requests with a page missing where some row sees a position have no context either.
__device__ __forceinline__ void check_pages(const Args& a, Requests& q) {
  const int all = 2 * q.tile[MAX_BATCH];
  for (int e = threadIdx.x; e < all; e += 256) {
    const int b = request_at(q.tile, a.batch, e >> 1);
    const Span sp = span_of(q.ctx[b], q.rows[b], a.window, a.sinks);
    const int t0 = base_of(sp, (e >> 1) - q.tile[b]) + 16 * (e & 1), slot = t0 >> a.page_log2;
    if (half_needed(a, sp, t0) &&
        (slot >= a.ld_table ||
         (uint32_t)a.table[(int64_t)b * a.ld_table + slot] >= (uint64_t)a.num_pages))
      q.status[b] = SV_ROW_BAD_PAGE;
  }
  __syncthreads();
  for (int b = threadIdx.x; b < a.batch; b += 256)
    if (q.status[b] == SV_ROW_BAD_PAGE) q.ctx[b] = -1;
  __syncthreads();
}

// Items by falling work, so that the shortest end the call: counted per level, then placed.
__device__ __forceinline__ void plan_items(const Args& a, const Requests& q, int* level) {
  constexpr int LEVELS = 64;
  const int tid = threadIdx.x, lane = tid & 63;
  for (int b = tid; b < a.batch; b += 256) a.status[b] = q.status[b];
  if (tid < LEVELS) level[tid] = 0;
  __syncthreads();
  const int blocks = q.block[MAX_BATCH], all = blocks * a.chunks;
  for (int pass = 0; pass < 2; ++pass) {
    for (int i = tid; i < all; i += 256) {
      const int blk = i / a.chunks, c = i - blk * a.chunks;
      const int b = request_at(q.block, a.batch, blk), rb = blk - q.block[b];
      int work = c == 0 ? 1 : 0;
      if (q.ctx[b] >= 0) {
        const uint32_t r0 = (uint32_t)rb * a.block_rows, R = (uint32_t)q.rows[b] * a.group;
        const int j0 = (int)(r0 / (uint32_t)a.group);
        const int j1 = (int)((min(r0 + a.block_rows, R) - 1) / (uint32_t)a.group);
        const int tiles = block_span(q.ctx[b], j0, j1, a.window, a.sinks).tiles;
        work = max(work, min(tiles - c * a.chunk_tiles, a.chunk_tiles));
      }
      if (work <= 0) continue;
      const int lv = LEVELS - 1 - (int)((int64_t)work * (LEVELS - 1) / a.chunk_tiles);
      if (pass == 0) {
        atomicAdd(&level[lv], 1);
      } else {
        const Item it = {b, rb, c, blk, q.row0[b], q.rows[b], q.ctx[b], q.tile[b]};
        // (places within a level come as they come: which workgroup computes an item changes
        // nothing in its result)
        a.items[atomicAdd(&level[lv], 1)] = it;
        if (c == 0) a.blocks[blk] = it;
      }
    }
    __syncthreads();
    if (pass == 0) {
      if (tid < 64) {
        const int x = level[lane];
        int sum = x;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const int y = __shfl_up(sum, d);
          if (lane >= d) sum += y;
        }
        level[lane] = sum - x;
        if (lane == 63) {
          a.head->items = sum;
          a.head->blocks = blocks;
        }
      }
      __syncthreads();
    }
  }
}

template <int BYTE>
__device__ __forceinline__ uint32_t widen(uint32_t word, float scale) {
  return __builtin_bit_cast(uint32_t,
                            __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, BYTE));
}

// A tile of one KV head in bf16, by a wave or a workgroup:
//   K [D/16][64][8]     step s, lane (n, g): token n, dims 16 s + 8 g ..
//   V [D/32][2][64][8]  dims' 32 i + n, tokens 16 u + 4 g + (0..3, 8..11)
// Positions that no row sees become 0.  A V block stored as NaN becomes 0 as well, and is
// noted, for it must not reach rows that do not see it (0 * NaN); a K block becomes NaN.
template <int D, int THREADS>
__device__ __forceinline__ void widen_tile(const Args& a, const Requests& q, int tile, int h) {
  const int me = threadIdx.x & (THREADS - 1);
  const int b = request_at(q.tile, a.batch, tile);
  const Span sp = span_of(q.ctx[b], q.rows[b], a.window, a.sinks);
  const int base = base_of(sp, tile - q.tile[b]);
  const int early = a.window > 0 ? min(a.sinks, sp.first) : 0;
  auto seen = [&](int t) { return t < sp.n && (t >= sp.first || t < early); };
  // its units: pages hold 16 tokens at least
  const uint8_t* unit[2];
  const int32_t* tab = a.table + (int64_t)b * a.ld_table;
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    const int t0 = base + 16 * hf, slot = t0 >> a.page_log2;
    const bool have = half_needed(a, sp, t0) && slot < a.ld_table;
    const uint32_t id = have ? (uint32_t)tab[slot] : 0xffffffffu;
    unit[hf] = id < (uint64_t)a.num_pages ? a.pages + ((int64_t)id * a.kv_heads + h) * a.unit : nullptr;
  }
  uint8_t* const dst = a.wide + ((int64_t)h * a.max_tiles + tile) * tile_bytes(D);
  const int P = a.page;

#pragma unroll
  for (int w0 = 0; w0 < D / 16 * 64; w0 += THREADS) {
    const int w = w0 + me, s = w >> 6, n = w & 31, g = w >> 5 & 1;
    const int t = base + n, at = t & (P - 1);
    const uint8_t* u = n < 16 ? unit[0] : unit[1];
    u32x4 y = {0, 0, 0, 0};
    if (u && seen(t)) {
      const uint32_t x = *(const uint32_t*)(u + at * (D / 2) + 8 * s + 4 * g);
      const uint32_t e = u[off_ks(P, D) + (at >> 3) * (D / 4) + (s / 2) * 8 + (at & 7)];
      const float sc = __builtin_bit_cast(float, e << 23);
      y[0] = widen<0>(x, sc);
      y[1] = widen<1>(x, sc);
      y[2] = widen<2>(x, sc);
      y[3] = widen<3>(x, sc);
      if (e == 255) y = u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
    }
    *(u32x4*)(dst + w * 16) = y;
  }
  // V: a pair of dims (a byte of a token) for 8 tokens, 4 of which lie side by side
  constexpr int B = D / 32;                   // bytes of a token in a 16th of the dims
#pragma unroll
  for (int w0 = 0; w0 < D / 2 * 4; w0 += THREADS) {
    const int w = w0 + me;
    if (D / 2 * 4 % THREADS != 0 && w >= D / 2 * 4) break;
    const int c = w % (D / 2), ug = w / (D / 2), u2 = ug >> 1, g = ug & 1;
    const uint8_t* u = u2 ? unit[1] : unit[0];
    const int n16 = 2 * c / (D / 16), byte = c % B;
    uint32_t x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = 0;
    if (u) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int t0 = base + 16 * u2 + 8 * hf + 4 * g, at = t0 & (P - 1);
        const uint8_t* v = u + off_v(P, D) + (at >> 3) * (4 * D) + n16 * (D / 4) + (at & 7) * B;
        const uint32_t e4 =
            *(const uint32_t*)(u + off_vs(P, D) + (at >> 3) * (D / 4) + (2 * c / 32) * 8 + (at & 7));
        uint32_t word[B];
        if constexpr (B == 2) {
          const u32x2 y = *(const u32x2*)v;
          word[0] = y[0];
          word[1] = y[1];
        } else {
#pragma unroll
          for (int i = 0; i < B / 4; ++i) {
            const u32x4 y = *(const u32x4*)(v + 16 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) word[4 * i + j] = y[j];
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t e = e4 >> 8 * k & 255u;
          uint32_t code;
          if constexpr (B == 8) {
            const uint32_t even = word[2 * k], more = word[2 * k + 1];
            code = (byte < 4 ? even : more) >> 8 * (byte & 3);
          }
          else if constexpr (B == 4) code = word[k] >> 8 * byte;
          else code = word[k / 2] >> 8 * (2 * (k & 1) + byte);
          if (e != 255 && seen(t0 + k)) x[4 * hf + k] = widen<0>(code, __builtin_bit_cast(float, e << 23));
        }
      }
    }
    u32x4 lo, hi;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      lo[k] = __builtin_amdgcn_perm(x[2 * k + 1], x[2 * k], 0x05040100u);
      hi[k] = __builtin_amdgcn_perm(x[2 * k + 1], x[2 * k], 0x07060302u);
    }
    u32x4* to = (u32x4*)(dst + TILE * D * 2) + ((c / 16 * 2 + u2) * 64 + 32 * g + 2 * c % 32);
    to[0] = lo;
    to[1] = hi;
  }
  if (me < 32) {
    const int n = me, t = base + n, at = t & (P - 1);
    const uint8_t* u = n < 16 ? unit[0] : unit[1];
    uint32_t m = 0;
    if (u && seen(t))
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
        m |= (uint32_t)(u[off_vs(P, D) + (at >> 3) * (D / 4) + k * 8 + (at & 7)] == 255) << k;
    const int64_t at_tile = (int64_t)h * a.max_tiles + tile;
    a.odd_blocks[at_tile * TILE + n] = (uint8_t)m;
    const uint32_t any = (uint32_t)__ballot(m != 0);
    if (n == 0) a.odd[at_tile] = any;
  }
}

// Workgroup 0 lists the items, the others widen the tiles of the requests' KV heads.
template <int D>
__global__ __launch_bounds__(256) void k_prompt_prepare(Args a) {
  __shared__ Requests q;
  __shared__ int level[64];
  find_requests(a, q);
  if (blockIdx.x == 0) {
    check_pages(a, q);
    plan_items(a, q, level);
    return;
  }
  // a tile of a KV head for each wave, or workgroup where there are few (64 prompts of 1 to 700
  // rows, 18,000 positions: 13.6 us, a workgroup each 18.7; one of 40 rows: 10.2 and 7.2)
  const int units = q.tile[MAX_BATCH] * a.kv_heads, first = (int)blockIdx.x - 1, step = (int)gridDim.x - 1;
  if (units <= step) {
    for (int u = first; u < units; u += step) widen_tile<D, 256>(a, q, u / a.kv_heads, u % a.kv_heads);
  } else {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int u = 4 * first + wave; u < units; u += 4 * step)
      widen_tile<D, 64>(a, q, u / a.kv_heads, u % a.kv_heads);
  }
}

template <typename T>
__device__ __forceinline__ float to_f32(T x) { return (float)x; }

template <int D, int OD, typename T>
struct Prompt {
  static constexpr int STEPS = D / 16, DT = OD / 32;
  static constexpr int K_WORDS = TILE * D * 2 / 16, V_WORDS = TILE * OD * 2 / 16,
                       WORDS = K_WORDS + V_WORDS;        // a tile in LDS, in 16 bytes
  // fp32 queries and weights are split into three bf16 terms (3 x 8 bits hold fp32's 24)
  static constexpr int NT = sizeof(T) == 4 ? 3 : 1;
  // (of fp32 rows at D=256 the last term lies in LDS: all three do not fit the registers)
  static constexpr int NR = NT == 3 && D == 256 ? 2 : NT;
  static constexpr int Q_LDS = STEPS * (NT - NR) * 64;    // 16-byte words of a wave
  // tiles weighed at a time: two where both fit the registers, but for D=64, whose short
  // prompts lose more to the half pairs at their ends (64 of 1 to 700 rows 79 us, in pairs 87;
  // four of 1,500 to 4,000 160 and 162)
  static constexpr int PAIR = NT == 1 && D == 128 ? 2 : 1;

  bf16x8 q[STEPS][NR];
  f32x16 o[DT];
  float l, m, mc, over;
  int pos;
  uint32_t poison;

  static __device__ __forceinline__ void split(float x, __bf16* t) {
    float r = x;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      t[i] = (__bf16)r;
      r -= (float)t[i];
    }
  }
  __device__ __forceinline__ void init(const Args& a, int row0, int ctx, int h, uint32_t r0, uint32_t R,
                                       u32x4* q_lds) {
    const int n = threadIdx.x & 31, g = threadIdx.x >> 5 & 1;
    const uint32_t r = min(r0 + n, R - 1);
    const uint32_t j = r / (uint32_t)a.group, hq = h * a.group + r - j * a.group;
    pos = ctx + (int)j;
    const T* src = (const T*)a.q + ((int64_t)row0 + j) * a.ld_q + (int64_t)hq * D + 8 * g;
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
      T x[8];
      __builtin_memcpy(x, src + 16 * st, sizeof(x));
      [[maybe_unused]] bf16x8 rest;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        __bf16 t[NT];
        if constexpr (NT == 1) t[0] = x[k];
        else split(to_f32<T>(x[k]), t);
#pragma unroll
        for (int u = 0; u < NR; ++u) q[st][u][k] = t[u];
        if constexpr (NR < NT) rest[k] = t[NT - 1];
      }
      if constexpr (NR < NT) q_lds[st * 64 + (threadIdx.x & 63)] = __builtin_bit_cast(u32x4, rest);
    }
    l = 0.f;
    m = over = -INFINITY;
    mc = -FAR;
    poison = 0;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int k = 0; k < 16; ++k) o[dt][k] = 0.f;
  }
  __device__ __forceinline__ bool sees(const Args& a, int t) const {
    const bool inside = (a.window == 0) | (t > pos - a.window) | (t < a.sinks);
    return inside & (t <= pos);
  }
  // Token of accumulator entry r, relative to the tile.
  static __device__ __forceinline__ int token(int g, int r) { return 8 * (r >> 2) + 4 * g + (r & 3); }

  __device__ __forceinline__ f32x16 scores(const u32x4* lds, const u32x4* q_lds) const {
    const int lane = threadIdx.x & 63;
    f32x16 y;
#pragma unroll
    for (int k = 0; k < 16; ++k) y[k] = 0.f;
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
      const bf16x8 kf = __builtin_bit_cast(bf16x8, lds[st * 64 + lane]);
      if constexpr (NR < NT)
        y = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            kf, __builtin_bit_cast(bf16x8, q_lds[st * 64 + lane]), y, 0, 0, 0);
#pragma unroll
      for (int u = NR - 1; u >= 0; --u)
        y = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, q[st][u], y, 0, 0, 0);
      // (or all operands are read ahead and do not fit the registers)
      if ((D == 256 || NT == 3) && st % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    }
    return y;
  }
  // PAIR tiles at lds; their first tokens; masked: some row does not see some token.
  __device__ __forceinline__ void step(const Args& a, const u32x4* lds, const u32x4* q_lds,
                                       const int (&base)[PAIR], bool masked, float c) {
    const int lane = threadIdx.x & 63, g = lane >> 5;
    f32x16 s[PAIR];
#pragma unroll
    for (int t = 0; t < PAIR; ++t) s[t] = scores(lds + t * WORDS, q_lds);
    // (the wave that has its scores goes before the one that makes them)
    if (D < 256) __builtin_amdgcn_s_setprio(1);
    if (masked) {
      asm volatile("");                       // (a branch: most tiles need no mask)
#pragma unroll
      for (int t = 0; t < PAIR; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[t][r] = sees(a, base[t] + token(g, r)) ? s[t][r] : -INFINITY;
    }
    float mx = fmaxf(s[0][0], s[0][1]);
#pragma unroll
    for (int r = 2; r < 16 * PAIR; r += 2)
      mx = fmaxf(fmaxf(mx, s[r / 16][r % 16]), s[r / 16][r % 16 + 1]);
    // (a first visible score raises -inf; a row that has seen nothing stays there)
    if (__any(mx > over)) {
      mx = fmaxf(mx, __shfl_xor(mx, 32));     // the other half of the row's tokens
      const float nm = fmaxf(m, mx);
      const float nc = __builtin_amdgcn_fmed3f(nm * c, -FAR, FAR);
      const float f = __builtin_amdgcn_exp2f(mc - nc);
      l *= f;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) o[dt] *= f;
      m = nm;
      mc = nc;
      over = nm + __builtin_fminf(RAISE / c, 3.4e38f);
    }
    bf16x8 p[PAIR][2][NT];
#pragma unroll
    for (int t = 0; t < PAIR; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][r], c, -mc));
        __bf16 x[NT];
        split(e, x);
#pragma unroll
        for (int u = 0; u < NT; ++u) p[t][r >> 3][u][r & 7] = x[u];
        if constexpr (NT > 1) l += e;
      }
    // (the sum of bf16 rows is that of the rounded weights: their errors cancel in the division)
    if constexpr (NT == 1)
#pragma unroll
      for (int t = 0; t < PAIR; ++t)
#pragma unroll
        for (int r = 0; r < 16; r += 2) {
          const bf16x2 two = {p[t][r >> 3][0][r & 7], p[t][r >> 3][0][(r & 7) + 1]};
          l = __builtin_amdgcn_fdot2_f32_bf16(two, bf16x2{(__bf16)1.f, (__bf16)1.f}, l, false);
        }
    if (D < 256) __builtin_amdgcn_s_setprio(0);
#pragma unroll
    for (int t = 0; t < PAIR; ++t)
#pragma unroll
      for (int u2 = 0; u2 < 2; ++u2)
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
          const bf16x8 vf =
              __builtin_bit_cast(bf16x8, lds[t * WORDS + K_WORDS + (dt * 2 + u2) * 64 + lane]);
#pragma unroll
          for (int u = NT - 1; u >= 0; --u)
            o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, p[t][u2][u], o[dt], 0, 0, 0);
          if (D == 256 || NT == 3) __builtin_amdgcn_sched_barrier(0);
        }
  }
  // V blocks stored as NaN: rows that see the token are NaN in the block's dims.
  __device__ __forceinline__ void note(const Args& a, int64_t place, int base) {
    for (uint32_t m = a.odd[place]; m; m &= m - 1) {
      const int t = __builtin_ctz(m);
      if (sees(a, base + t)) poison |= a.odd_blocks[place * TILE + t];
    }
  }
};

// The wave's loads straight to LDS have arrived: before a barrier that hands them to the other
// waves (the loads name no register that a later use would make the compiler wait for).
__device__ __forceinline__ void direct_loads_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

template <int D, int OD, int WAVES, int PER_SIMD, typename T>
__global__ __launch_bounds__(64 * WAVES, PER_SIMD) void k_prompt(Args a) {
  using A = Prompt<D, OD, T>;
  constexpr int PARTS = D / OD;               // workgroups that share a block's dims
  // tiles in LDS between two barriers, twice (160 KiB per compute unit; the more, the better:
  // four prompts of 1,500 to 4,000 rows at D=256 with two 1,096 us, with one 1,299)
  constexpr int STAGE = D < 256 ? WAVES / 2 : sizeof(T) == 2 ? WAVES / 4 : 1;
  constexpr int WORDS = A::WORDS, LOADS = STAGE * WORDS / (64 * WAVES);
  __shared__ u32x4 lds[2][STAGE * WORDS], q_lds[A::Q_LDS ? WAVES : 1][A::Q_LDS ? A::Q_LDS : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int of = blockIdx.x % PARTS, hit = blockIdx.x / PARTS;
  const int it = hit / a.kv_heads, h = hit - it * a.kv_heads;
  const Item item = a.items[it];              // (anything, past the last)
  if (it >= a.head->items) return;
  const int row0 = item.row0, rows = item.rows, ctx = item.ctx;
  // (rows * heads of a call are less than 2^31)
  const uint32_t R = (uint32_t)rows * a.group, r0 = (uint32_t)item.rb * a.block_rows;
  const uint32_t rw = r0 + wave * 32;         // the wave's first row
  const int n = lane & 31, g = lane >> 5;
  auto row_out = [&](uint32_t r) {
    const uint32_t j = r / (uint32_t)a.group, hq = h * a.group + r - j * a.group;
    return (T*)a.out + ((int64_t)row0 + j) * a.ld_out + (int64_t)hq * D + of * OD;
  };
  if (ctx < 0) {                              // the request's rows are NaN
    if (item.chunk > 0 || rw + n >= R) return;
    T* const dst = row_out(rw + n);
    for (int i = 0; i < OD / 2; ++i) dst[g * (OD / 2) + i] = (T)__builtin_nanf("");
    return;
  }
  const int j0 = (int)(r0 / (uint32_t)a.group);
  const int j1 = (int)((min(r0 + a.block_rows, R) - 1) / (uint32_t)a.group);
  const Span all = span_of(ctx, rows, a.window, a.sinks);
  const Span sp = block_span(ctx, j0, j1, a.window, a.sinks);
  const int begin = item.chunk * a.chunk_tiles, end = min(sp.tiles, begin + a.chunk_tiles);
  const bool whole = sp.tiles <= a.chunk_tiles;
  const float c = a.scale * LOG2E;
  const int64_t first = (int64_t)h * a.max_tiles + item.tile;
  // where tile i of the block lies in its widened form
  auto place = [&](int i) {
    const int t = i < sp.early ? i : i - sp.early + sp.tile0;
    return first + (t < all.early ? t : t - all.tile0 + all.early);
  };
  // positions of the wave's rows
  const int w0 = ctx + (int)(min(rw, R - 1) / (uint32_t)a.group);
  const int w1 = ctx + (int)(min(rw + 31, R - 1) / (uint32_t)a.group);
  const bool live = rw < R;
  auto masked = [&](int base) {
    return base + TILE - 1 > w0 || (a.window > 0 && base <= w1 - a.window && base + TILE > a.sinks);
  };

  // the next tiles go straight to LDS, 1 KiB per wave and instruction
  auto ask = [&](int i, int buf) {
    uint32_t mine = lane * 16;
    asm volatile("" : "+v"(mine));            // (or its sum with the base is kept, and no scalar any more)
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
      const int w = (k * WAVES + wave) * 64, t = w / WORDS, x = w - t * WORDS;
      // (scalar, so that a load's address costs no vector arithmetic)
      const uint32_t at = (uint32_t)__builtin_amdgcn_readfirstlane((int)place(min(i + t, end - 1)));
      const uint8_t* src = a.wide + ((int64_t)at * tile_bytes(D) +
                                     (x + (x < A::K_WORDS ? 0 : of * A::V_WORDS)) * 16);
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src + mine),
                                       (__attribute__((address_space(3))) void*)(lds[buf] + w), 16, 0, 0);
    }
  };
  ask(begin, 0);
  A x;
  u32x4* const my_q = q_lds[A::Q_LDS ? wave : 0];
  x.init(a, row0, ctx, h, rw, R, my_q);
  uint32_t some_odd = 0;
  for (int i = begin + (int)threadIdx.x; i < end; i += 64 * WAVES) some_odd |= a.odd[place(i)];
  const bool odd = __syncthreads_or(some_odd != 0);
  direct_loads_done();
  __syncthreads();
  int buf = 0;
  for (int i = begin; i < end; i += STAGE) {
    if (i + STAGE < end) ask(i + STAGE, buf ^ 1);
#pragma unroll
    for (int t = 0; t < STAGE; t += A::PAIR) {
      int base[A::PAIR];
      bool some = false, hide = false;
#pragma unroll
      for (int k = 0; k < A::PAIR; ++k) {
        // (behind the last tile lies that tile once more: no row sees it there)
        base[k] = i + t + k < end ? base_of(sp, i + t + k) : 0x7fffff00;
        some |= base[k] <= w1;
        hide |= masked(base[k]);
      }
      if (live && some) {
        x.step(a, lds[buf] + t * WORDS, my_q, base, hide, c);
        if (odd)
          for (int k = 0; k < A::PAIR; ++k)
            if (i + t + k < end) x.note(a, place(i + t + k), base[k]);
      }
    }
    buf ^= 1;
    direct_loads_done();
    __syncthreads();
  }

  const int64_t slot = (((int64_t)item.block * a.kv_heads + h) * a.chunks + item.chunk) * a.block_rows;
  float* const part = a.part + slot * D + of * OD;
  float* const stat = a.part + (int64_t)a.max_blocks * a.kv_heads * a.chunks * a.block_rows * D + slot * 2;
  const float sum = x.l + __shfl_xor(x.l, 32);
  int ln = lane & 31;
  asm volatile("" : "+v"(ln));                // (or where the row lies takes registers in the loop)
  const uint32_t r = rw + ln;
  if (r >= R) return;
  T* const dst = row_out(r);
  const float inv = 1.f / sum;
  const int local = (int)(r - r0);
#pragma unroll
  for (int dt = 0; dt < A::DT; ++dt) {
    const bool nan = x.poison >> (of * A::DT + dt) & 1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = nan ? __builtin_nanf("") : x.o[dt][4 * k + e];
      const int dim = 32 * dt + 8 * k + 4 * g;
      if (whole) {
        T z[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = (T)(y[e] * inv);
        __builtin_memcpy(dst + dim, z, sizeof(z));
      } else {
        __builtin_memcpy(part + (int64_t)local * D + dim, y, sizeof(y));
      }
    }
  }
  if (!whole && g == 0 && of == 0) {
    stat[local * 2] = x.mc;
    stat[local * 2 + 1] = sum;
  }
}

// Joins the chunks of blocks that have several: 16 threads per row.
template <int D, typename T>
__global__ __launch_bounds__(256) void k_prompt_join(Args a) {
  constexpr int E = D / 16;
  const int per = a.block_rows / 16;
  const int local = (int)(blockIdx.x % per) * 16 + (threadIdx.x >> 4), e0 = (threadIdx.x & 15) * E;
  const int hb = blockIdx.x / per, h = hb % a.kv_heads, bl = hb / a.kv_heads;
  if (bl >= a.head->blocks) return;
  const Item blk = a.blocks[bl];
  if (blk.ctx < 0) return;
  const int row0 = blk.row0, rows = blk.rows;
  const uint32_t R = (uint32_t)rows * a.group, r0 = (uint32_t)blk.rb * a.block_rows, r = r0 + local;
  const int j0 = (int)(r0 / (uint32_t)a.group);
  const int j1 = (int)((min(r0 + a.block_rows, R) - 1) / (uint32_t)a.group);
  const int tiles = block_span(blk.ctx, j0, j1, a.window, a.sinks).tiles;
  const int n = (tiles + a.chunk_tiles - 1) / a.chunk_tiles;
  if (n < 2 || r >= R) return;
  const int64_t slot = ((int64_t)bl * a.kv_heads + h) * a.chunks * a.block_rows + local;
  const float* part = a.part + slot * D + e0;
  const float* stat = a.part + (int64_t)a.max_blocks * a.kv_heads * a.chunks * a.block_rows * D + slot * 2;
  float m = -INFINITY;
  for (int k = 0; k < n; ++k) m = fmaxf(m, stat[(int64_t)k * a.block_rows * 2]);
  float acc[E] = {}, sum = 0.f;
  for (int k = 0; k < n; ++k) {
    const float mk = stat[(int64_t)k * a.block_rows * 2];
    const float w = mk == m ? 1.f : __builtin_amdgcn_exp2f(mk - m);
    sum += w * stat[(int64_t)k * a.block_rows * 2 + 1];
    float y[E];
    __builtin_memcpy(y, part + (int64_t)k * a.block_rows * D, sizeof(y));
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = __builtin_fmaf(y[e], w, acc[e]);
  }
  const uint32_t j = r / (uint32_t)a.group, hq = h * a.group + r - j * a.group;
  T z[E];
#pragma unroll
  for (int e = 0; e < E; ++e) z[e] = (T)(acc[e] / sum);
  __builtin_memcpy((T*)a.out + ((int64_t)row0 + j) * a.ld_out + (int64_t)hq * D + e0, z, sizeof(z));
}

// ---- host side

struct Plan {
  int waves, block_rows, max_blocks, chunks, chunk_tiles;
  int64_t max_tiles;
  size_t blocks, items, odd, odd_blocks, wide, part, bytes;
};

static size_t round256(size_t x) { return (x + 255) / 256 * 256; }

static bool plan_of(int dtype, int batch, int total_rows, int heads, int kv_heads, int d,
                    int max_context, int64_t total_context, int window, int sinks, Plan& p) {
  const int64_t R = (int64_t)total_rows * (heads / kv_heads);
  // Four waves per workgroup, two workgroups per compute unit, so that one's start and end
  // run beside the other's products; or eight, which share a tile's way to LDS, for bf16 calls
  // of many workgroups and long contexts.  (us with eight waves and with four, by the call's rows
  // of all KV heads over 256.  Eight: one prompt of 15,991 rows, 2,000: 1,850 and 1,945; four of
  // 1,500 to 4,000, 1,150: 296 and 301 to 306.  Four: eight of 800 to 2,000 over 16 KV heads, 580:
  // 108 and 102; two of 150 to 600 after 8,000 to 30,000 positions, 56: 287 and 251; 64 of 1 to
  // 700, 2,150, short: equal; eight fp32 ones with a window: 203 and 172.)
  p.waves = 8;
  int64_t blocks = 0;
  for (;; p.waves = 4) {
    p.block_rows = 32 * p.waves;
    blocks = (R + (int64_t)batch * (p.block_rows - 1)) / p.block_rows;
    if (p.waves == 4 ||
        (dtype == SV_BF16 && R * kv_heads >= 1024 * 256 && total_context >= (int64_t)batch * 1024))
      break;
  }
  // tiles of all requests, and of one
  int64_t tiles = total_context / TILE + batch, one = max_context / TILE + 1;
  if (window > 0) {
    const int64_t more = (int64_t)window / TILE + (sinks + TILE - 1) / TILE + 3;
    const int64_t seen = total_rows / TILE + batch * more;
    if (seen < tiles) tiles = seen;
    const int64_t block_seen = p.block_rows / TILE + more;
    if (block_seen < one) one = block_seen;
  }
  p.max_tiles = tiles;
  int64_t chunks = 1;
  const int64_t wide = blocks * kv_heads;
  if (wide < 512) chunks = (512 + wide - 1) / wide;
  int64_t ct = (one + chunks - 1) / chunks;
  if (ct < 16) ct = 16;
  chunks = (one + ct - 1) / ct;
  p.chunks = (int)chunks;
  p.chunk_tiles = (int)ct;
  // (a launch has less than 2^32 threads, two workgroups per block at D=256; the join is launched
  // only where blocks are few)
  if (wide * chunks * (d == 256 ? 2 : 1) * (64 * p.waves) >= (1ll << 32) || tiles * kv_heads >= (1ll << 24))
    return false;
  p.max_blocks = (int)blocks;
  size_t at = round256(sizeof(Head));
  p.blocks = at;
  at += round256((size_t)blocks * sizeof(Item));
  p.items = at;
  at += round256((size_t)(blocks * chunks) * sizeof(Item));
  p.odd = at;
  at += round256((size_t)(tiles * kv_heads) * 4);
  p.odd_blocks = at;
  at += round256((size_t)(tiles * kv_heads) * TILE);
  p.wide = at;
  at += (size_t)(tiles * kv_heads) * tile_bytes(d);
  p.part = at;
  if (chunks > 1) at += (size_t)(wide * chunks * p.block_rows) * (d + 2) * sizeof(float);
  p.bytes = at;
  return true;
}

static bool sizes_ok(int dtype, int batch, int total_rows, int heads, int kv_heads, int d,
                     int max_context, int64_t total_context, int window, int sinks) {
  return (dtype == SV_F32 || dtype == SV_BF16) && batch >= 1 && batch <= MAX_BATCH &&
         total_rows >= 1 && kv_heads >= 1 && heads >= kv_heads && heads % kv_heads == 0 &&
         heads <= 1024 && dim_ok(d) && (int64_t)total_rows * heads < (1ll << 31) &&
         max_context >= 1 && max_context <= (1 << 30) && total_context >= 1 &&
         total_context <= (1ll << 30) && window >= 0 && window <= (1 << 30) && sinks >= 0 &&
         sinks <= (1 << 30);
}

template <int D, int OD, typename T>
static int launch(const Args& a, const Plan& p, hipStream_t s) {
  constexpr int PER_SIMD = sizeof(T) == 4 && D == 256 ? 1 : 2;
  const int64_t units = p.max_tiles * a.kv_heads;
  const dim3 prepare(1 + (uint32_t)(units < 1024 ? units : 1024));
  hipLaunchKernelGGL((k_prompt_prepare<D>), prepare, dim3(256), 0, s, a);
  if (hipGetLastError() != hipSuccess) return SV_ERR_LAUNCH;
  const uint32_t wide = (uint32_t)(p.max_blocks * a.kv_heads);
  const dim3 grid(wide * p.chunks * (D / OD));
  if (p.waves == 4) {
    hipLaunchKernelGGL((k_prompt<D, OD, 4, PER_SIMD, T>), grid, dim3(256), 0, s, a);
  } else {
    if constexpr (sizeof(T) == 2)
      hipLaunchKernelGGL((k_prompt<D, OD, 8, PER_SIMD, T>), grid, dim3(512), 0, s, a);
  }
  if (hipGetLastError() != hipSuccess) return SV_ERR_LAUNCH;
  if (p.chunks > 1) {
    hipLaunchKernelGGL((k_prompt_join<D, T>), dim3(wide * (a.block_rows / 16)), dim3(256), 0, s, a);
    if (hipGetLastError() != hipSuccess) return SV_ERR_LAUNCH;
  }
  return SV_OK;
}

}  // namespace prompt
}  // namespace svk

using namespace svk;

extern "C" {

size_t spec_kv_prompt_workspace_bytes(int dtype, int batch, int total_rows, int heads, int kv_heads,
                                      int head_dim, int max_context, int64_t total_context,
                                      int window, int sinks) {
  prompt::Plan p;
  if (!prompt::sizes_ok(dtype, batch, total_rows, heads, kv_heads, head_dim, max_context, total_context,
                        window, sinks) ||
      !prompt::plan_of(dtype, batch, total_rows, heads, kv_heads, head_dim, max_context, total_context,
                       window, sinks, p))
    return 0;
  return p.bytes;
}

int spec_kv_prompt_attention(const void* q, int64_t ld_q, int dtype, const int32_t* cu_seqlens,
                             const int32_t* context_lens, int batch, int total_rows, int heads,
                             int kv_heads, int head_dim, const void* pages, int64_t num_pages,
                             int page_size, const int32_t* page_table, int64_t ld_table,
                             int max_context, int64_t total_context, float scale, int window,
                             int sinks, void* out, int64_t ld_out, int32_t* status, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (!q || !cu_seqlens || !context_lens || !pages || !page_table || !out || !status)
    return SV_ERR_NULL;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  prompt::Plan p;
  if (!prompt::sizes_ok(dtype, batch, total_rows, heads, kv_heads, head_dim, max_context, total_context,
                        window, sinks) ||
      !page_ok(page_size) || num_pages < 1 || num_pages > 0x7fffffff || ld_table < 1 ||
      ld_table > (1 << 30) / page_size || ld_q < (int64_t)heads * head_dim ||
      ld_out < (int64_t)heads * head_dim || !(scale > 0.f) || !(scale <= 2.0e38f) ||
      !aligned16(pages) ||
      !prompt::plan_of(dtype, batch, total_rows, heads, kv_heads, head_dim, max_context, total_context,
                       window, sinks, p))
    return SV_ERR_SHAPE;
  if (!workspace || !aligned16(workspace)) return SV_ERR_NULL;
  if (p.bytes > workspace_bytes) return SV_ERR_WORKSPACE;
  // (a row's queries are read by several workgroups, at no fixed time before its result is written)
  const int64_t size = dtype == SV_F32 ? 4 : 2;
  if (rows_overlap(q, ld_q * size, out, ld_out * size, total_rows, heads * (int64_t)head_dim * size))
    return SV_ERR_SHAPE;
  prompt::Args a;
  a.q = q;
  a.ld_q = ld_q;
  a.cu = cu_seqlens;
  a.ctx = context_lens;
  a.batch = batch;
  a.total_rows = total_rows;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.group = heads / kv_heads;
  a.pages = (const uint8_t*)pages;
  a.num_pages = num_pages;
  a.page = page_size;
  a.page_log2 = __builtin_ctz((unsigned)page_size);
  a.unit = (int)unit_bytes(page_size, head_dim);
  a.table = page_table;
  a.ld_table = ld_table;
  a.max_context = max_context;
  a.total_context = total_context;
  a.scale = scale;
  a.window = window;
  a.sinks = sinks;
  a.out = out;
  a.ld_out = ld_out;
  a.status = status;
  a.block_rows = p.block_rows;
  a.max_blocks = p.max_blocks;
  a.chunks = p.chunks;
  a.chunk_tiles = p.chunk_tiles;
  a.max_tiles = p.max_tiles;
  uint8_t* w = (uint8_t*)workspace;
  a.head = (prompt::Head*)w;
  a.blocks = (prompt::Item*)(w + p.blocks);
  a.items = (prompt::Item*)(w + p.items);
  a.odd = (uint32_t*)(w + p.odd);
  a.odd_blocks = w + p.odd_blocks;
  a.wide = w + p.wide;
  a.part = (float*)(w + p.part);
  hipStream_t s = (hipStream_t)stream;
  if (dtype == SV_BF16) {
    if (head_dim == 64) return prompt::launch<64, 64, __bf16>(a, p, s);
    if (head_dim == 128) return prompt::launch<128, 128, __bf16>(a, p, s);
    return prompt::launch<256, 128, __bf16>(a, p, s);
  }
  if (head_dim == 64) return prompt::launch<64, 64, float>(a, p, s);
  if (head_dim == 128) return prompt::launch<128, 128, float>(a, p, s);
  return prompt::launch<256, 128, float>(a, p, s);
}

}  // extern "C"
