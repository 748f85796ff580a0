// kvbudget.hip -- a cache held to a budget of positions (include/specverify_cache.h states
// the operators):
//   spec_kv_attention_weights   the attention weight that cached positions get
//   spec_kv_evict               positions of the least weight leave the cache
//
// No float atomics: every position's weight is summed by one workgroup in a fixed order, and
// which positions stay follows from the weights and positions alone.

#include "kv_common.h"

namespace svk {
namespace budget {

// ------------------------------------------------------------------ weights
//
// W[b][h][t] = in[b][h][t] + sum over the counted rows j and the query heads of KV head h of
//   exp(scale q.k_t - m) / sum_u exp(scale q.k_u - m)
// The divisor needs every score of a row before the first weight, so the scores are made
// twice: once for the rows' maxima and sums, once for the weights.  (Kept instead, they would
// take R numbers per position, more than the position's codes from R = 16 on.)
//
// A workgroup of 4 waves takes a chunk of one KV head's context and all R = rows * G query
// rows of it, whose operands lie in LDS; its waves take the tiles of 32 tokens in turn.
// Scores are made with v_mfma_f32_16x16x32_bf16, K widened from its codes in registers.  For
// the sums as S^T[token][row] = K Q^T: a lane holds one row's scores for 8 tokens, and goes over
// the tiles for each 16 MT rows with the row's statistics in registers.  For the weights as
// S[row][token] = Q K^T: a lane holds two tokens' scores for 4 MT rows, and goes over the rows of
// each tile with the tokens' weights in registers (with S^T there too, sums over 16 lanes
// for each of 8 tokens, 64 requests of 7 rows over 512 to 16,384 positions took 123 us, so 113).
// Where a request is one chunk (short contexts) both passes are one launch.  fp32 queries go in
// as three bf16 terms, exactly; nothing is rounded further.
//
// What bounds it: vector instructions, 64 % of the first pass's time and 59 % of the second's,
// beside HBM at 3.8 and 3.4 TB/s: 51 + 62 us for 64 requests of 7 rows over 512 to 16,384
// positions (32 heads over 8, D=128).  They are widening, exponentials, and scalars kept in lanes
// of vector registers for want of scalar ones (74 and 95 of them here, 181 to 335 with four
// row tiles): ten to twenty reads of such lanes per tile, and 58 with 37 writes for a block of 64
// rows that is masked.  Four requests of 64 rows over 1,500 to 4,000 positions, 26 + 31 us: 1.4
// waves per SIMD whose reads of queries from LDS and exponentials follow one another (smaller
// chunks give more waves, and more queries to fetch: no faster; eight waves per workgroup 73 us
// against 58 for the call).

constexpr int TILE = 32, SUB = 64;            // tokens of a tile; tiles whose pages a wave looks up at once
// Waves of a workgroup: eight where it does both passes (64 requests over 100 to 1,000 positions
// 21 us; before the weights went over rows in the lane 22.5, four waves 23.7, sixteen 31, two
// launches 30).
constexpr int waves_of(bool both) { return both ? 8 : 4; }
constexpr float LOG2E = 1.44269504088896340736f;
// the rounded product of maximum and scale, from which exponents are counted, is held within
// +-FAR: past it weights become infinite, or all 0, and their row adds nothing
constexpr float FAR = 1073741824.0f;          // 2^30

struct WeightArgs {
  const void* q;
  int64_t ld_q;
  const int32_t *cu, *ctx, *counts;
  int batch, total_rows, max_k, heads, kv_heads, group;
  float inv_group;
  const uint8_t* pages;
  int64_t num_pages;
  int page, page_log2, unit;
  const int32_t* table;
  int64_t ld_table;
  int max_context;
  float scale;
  int window, sinks;
  const float* in;
  float* out;
  int64_t ld_w;
  int32_t* status;
  int chunks, chunk_tiles, max_rows;          // chunks of a request at most; R at most
  int group_rows;                             // rows whose queries lie in LDS at once
  float* stats;                               // [batch][kv_heads][chunks][max_rows][2]
  int gap_blocks;                             // blocks per KV head that copy what no row sees
};

struct Request {
  int row0, rows, count, ctx, status;
};
__device__ __forceinline__ Request request_of(const WeightArgs& a, int b) {
  Request r;
  const int c0 = a.cu[b], c1 = a.cu[b + 1], cx = a.ctx[b];
  const int cnt = a.counts ? a.counts[b] : c1 - c0;
  const int broken = first_broken(a.cu, a.batch, a.total_rows);
  r.row0 = c0;
  r.rows = c1 - c0;
  r.count = cnt;
  r.ctx = cx;
  r.status = SV_ROW_OK;
  if (b >= broken || r.rows < 1 || r.rows > a.max_k + 1) r.status = SV_ROW_BAD_K;
  else if (cx < 0 || (int64_t)cx + r.rows > a.max_context || cnt < 0 || cnt > r.rows)
    r.status = SV_ROW_BAD_PARAM;
  return r;
}

// Tiles that the rows see: the first `early` of the sequence, then those from tile0 on.
struct Span {
  int n, first, early, tile0, tiles;
};
__device__ __forceinline__ Span span_of(const WeightArgs& a, const Request& r) {
  Span s;
  s.n = r.ctx + r.rows;
  s.first = a.window > 0 ? max(0, r.ctx - a.window + 1) : 0;
  s.tile0 = s.first / TILE;
  s.early = a.window > 0 ? min((a.sinks + TILE - 1) / TILE, s.tile0) : 0;
  s.tiles = s.early + (s.n - 1) / TILE - s.tile0 + 1;
  return s;
}
__device__ __forceinline__ int base_of(const Span& s, int i) {
  return (i < s.early ? i : i - s.early + s.tile0) * TILE;
}
// Whether a page that the rows need is missing; all lanes of a wave take part.
__device__ __forceinline__ bool pages_missing(const WeightArgs& a, const Span& sp, int b) {
  const int32_t* tab = a.table + (int64_t)b * a.ld_table;
  bool bad = false;
  for (int s = threadIdx.x & 63; s <= (sp.n - 1) >> a.page_log2; s += 64) {
    const int t0 = s << a.page_log2, t1 = t0 + a.page;
    if (t1 > sp.first || (a.window > 0 && t0 < a.sinks))
      bad |= s >= a.ld_table || (uint32_t)tab[s] >= (uint64_t)a.num_pages;
  }
  return __any(bad);
}
// Whether some row sees a position of the 16 from t0 on.
__device__ __forceinline__ bool half_needed(const WeightArgs& a, const Span& s, int t0) {
  return t0 < s.n && (t0 + 16 > s.first || (a.window > 0 && t0 < a.sinks));
}

template <int BYTE>
__device__ __forceinline__ uint32_t widen(uint32_t word, float scale) {
  return __builtin_bit_cast(uint32_t,
                            __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, BYTE));
}

template <int D>
struct KTile {
  uint32_t k[2][D / 32], ks[2][(D + 127) / 128];   // per half of 16 tokens: token n, D/4 dims
};

template <int D, int MT, typename T>
struct Weights {
  static constexpr int STEPS = D / 32, KB = (D + 127) / 128;
  // fp32 queries are split into three bf16 terms (3 x 8 bits hold fp32's 24)
  static constexpr int NT = sizeof(T) == 4 ? 3 : 1;
  static constexpr int ROWS = 16 * MT;
  static constexpr int Q_WORDS = MT * STEPS * NT * 64;      // 16-byte words of 16 MT rows

  // The operands of rows r0 .. r0 + 16 tiles - 1 in LDS, [row tile][step][term][lane].
  static __device__ __forceinline__ void put_q(const WeightArgs& a, bf16x8* q, const Request& rq,
                                               int h, int r0, int tiles, int R, int wave, int waves) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    for (int at = wave; at < tiles * STEPS; at += waves) {
      const int mt = at / STEPS, s = at % STEPS;
      const int r = min(r0 + mt * 16 + n, R - 1);
      const int j = r / a.group, hq = h * a.group + r - j * a.group;
      T x[8];
      __builtin_memcpy(x, (const T*)a.q + (int64_t)(rq.row0 + j) * a.ld_q + hq * D + g * (D / 4) + 8 * s,
                       sizeof(x));
      bf16x8 y[NT];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float rest = (float)x[k];
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          y[u][k] = (__bf16)rest;
          rest -= (float)y[u][k];
        }
      }
#pragma unroll
      for (int u = 0; u < NT; ++u) q[(at * NT + u) * 64 + lane] = y[u];
    }
  }

  // Pages of 64 tiles from `from` on: lane i holds those of tile from + i (its two halves).
  struct Pages {
    int id[2], first;
    __device__ __forceinline__ bool ask(const WeightArgs& a, const Span& sp, const int32_t* tab,
                                        int from, int end) {
      const int i = from + (threadIdx.x & 63);
      bool bad = false;
      first = from;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int t0 = base_of(sp, min(i, end - 1)) + 16 * hf, slot = t0 >> a.page_log2;
        const bool need = i < end && half_needed(a, sp, t0);
        const bool have = need && slot < a.ld_table;
        id[hf] = tab[have ? slot : 0];
        const bool in_pool = have && (uint32_t)id[hf] < (uint64_t)a.num_pages;
        bad |= need && !in_pool;
        if (!in_pool) id[hf] = 0;
      }
      return __any(bad);
    }
  };
  static __device__ __forceinline__ void fetch(const WeightArgs& a, KTile<D>& t, const uint8_t* pool,
                                               const Pages& id, const Span& sp, int i) {
    const uint32_t lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int base = base_of(sp, i);
    const uint32_t at_k = n * (D / 2) + g * (D / 8);
    const uint32_t at_s = off_ks(a.page, D) + (n >> 3) * (D / 4) + (g * (D / 4) / 32) * 8 + (n & 7);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const uint32_t page = (uint32_t)__builtin_amdgcn_readlane(id.id[hf], i - id.first);
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(pool + (uint64_t)page * ((uint32_t)a.unit * (uint32_t)a.kv_heads)), 0, a.unit, 0x00020000);
      const int tb = (base + 16 * hf) & (a.page - 1);
      if constexpr (D == 64) {
        const u32x2 k = __builtin_amdgcn_raw_buffer_load_b64(r, at_k, tb * (D / 2), 0);
        t.k[hf][0] = k[0];
        t.k[hf][1] = k[1];
      } else {
#pragma unroll
        for (int x = 0; x < D / 128; ++x) {
          const u32x4 k = __builtin_amdgcn_raw_buffer_load_b128(r, at_k + 16 * x, tb * (D / 2), 0);
#pragma unroll
          for (int j = 0; j < 4; ++j) t.k[hf][4 * x + j] = k[j];
        }
      }
#pragma unroll
      for (int x = 0; x < KB; ++x)
        t.ks[hf][x] = __builtin_amdgcn_raw_buffer_load_b8(r, at_s + 8 * x, tb * (D / 32), 0);
    }
  }

  // A tile's scores with 16 MT rows, -inf where a row (at pos_of(row tile, entry)) does not see
  // the token.  For the sums entry i of s[hf][mt] is token 16 hf + 4 g + i with row 16 mt + n,
  // and tokens of a block stored as NaN get NaN (their row then adds nothing); for the WEIGHTS
  // it is token 16 hf + n with row 16 mt + 4 g + i, and such tokens get -inf.
  template <bool WEIGHTS, typename Pos>
  static __device__ __forceinline__ void scores(const WeightArgs& a, const KTile<D>& t, const bf16x8* q,
                                                f32x4 (&s)[2][MT], int base, bool masked, Pos&& pos_of) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    int ql = lane;
    asm volatile("" : "+v"(ql));              // (or the reads move out of the loop, into registers)
    float sc[2][KB];
    uint32_t top = 0;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int x = 0; x < KB; ++x) {
        sc[hf][x] = __builtin_bit_cast(float, t.ks[hf][x] << 23);
        top = max(top, t.ks[hf][x]);
      }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) s[hf][mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
      u32x4 k[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint32_t x = t.k[hf][st];
        const float f = sc[hf][st / 4];
        k[hf][0] = widen<0>(x, f);
        k[hf][1] = widen<1>(x, f);
        k[hf][2] = widen<2>(x, f);
        k[hf][3] = widen<3>(x, f);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int u = NT - 1; u >= 0; --u) {
          const bf16x8 y = q[((mt * STEPS + st) * NT + u) * 64 + ql];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const bf16x8 x = __builtin_bit_cast(bf16x8, k[hf]);
            s[hf][mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(WEIGHTS ? y : x, WEIGHTS ? x : y,
                                                                s[hf][mt], 0, 0, 0);
          }
        }
    }
    if (__any(top == 255u)) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        bool o = false;
#pragma unroll
        for (int x = 0; x < KB; ++x) o |= t.ks[hf][x] == 255u;
        uint64_t m = __ballot(o);             // bit 16 g + n: token n
        m |= m >> 32;
        m |= m >> 16;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (m >> (WEIGHTS ? n : 4 * g + r) & 1)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) s[hf][mt][r] = WEIGHTS ? -INFINITY : __builtin_nanf("");
      }
    }
    if (masked) {
      asm volatile("");                       // (a branch: most tiles need no mask)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int pos = pos_of(mt, i);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int tok = base + 16 * hf + (WEIGHTS ? n : 4 * g + i);
            const bool inside = (a.window == 0) | (tok > pos - a.window) | (tok < a.sinks);
            if (!(inside & (tok <= pos))) s[hf][mt][i] = -INFINITY;
          }
        }
    }
  }
};

// Adds a part of a row's sum, counted from om, to one counted from m.
__device__ __forceinline__ void join(float& m, float& sum, float om, float osum) {
  const float nm = fmaxf(m, om);
  sum = sum * (m == nm ? 1.f : __builtin_amdgcn_exp2f(m - nm)) +
        osum * (om == nm ? 1.f : __builtin_amdgcn_exp2f(om - nm));
  m = nm;
}

// PASS 1: statistics, 2: weights, 3: both (a request is one chunk).  ONE: a request has at
// most 16 MT rows.
template <int D, int MT, bool ONE, int PASS, typename T>
__global__ __launch_bounds__(64 * waves_of(PASS == 3), PASS != 3 || D == 256 || MT == 4 ? 2 : 4)
void k_weights(WeightArgs a) {
  using A = Weights<D, MT, T>;
  constexpr int WAVES = waves_of(PASS == 3);
  constexpr int ROWS = A::ROWS, DEPTH = 2;    // tiles on their way
  // the queries of a.group_rows rows, then their waves' statistics or their maxima and
  // reciprocal sums
  extern __shared__ __align__(16) uint8_t smem[];
  bf16x8* const q = (bf16x8*)smem;
  f32x2* const part = (f32x2*)(smem + (size_t)a.group_rows * D * 2 * A::NT);   // [wave][row]
  f32x2* const fin = part + (PASS & 1 ? WAVES * a.group_rows : 0);             // [row]
  __shared__ int any_bad;
  __shared__ float acc[PASS & 2 ? (PASS == 3 ? 4 * WAVES : SUB) * TILE : 1];      // weights of a chunk
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int status_blocks = PASS & 1 ? (a.batch + WAVES - 1) / WAVES : 0;
  if ((int)blockIdx.x < status_blocks) {      // a request's status, a wave each
    const int b = (int)blockIdx.x * WAVES + wave;
    if (b >= a.batch) return;
    const Request rq = request_of(a, b);
    int st = rq.status;
    if (st == SV_ROW_OK && pages_missing(a, span_of(a, rq), b)) st = SV_ROW_BAD_PAGE;
    if (lane == 0) a.status[b] = st;
    return;
  }
  int it = (int)blockIdx.x - status_blocks;
  const int items = a.batch * a.kv_heads * a.chunks;
  if (it >= items) {                          // positions that no row sees keep what they have
    it -= items;
    const int share = it % a.gap_blocks, bh = it / a.gap_blocks, b = bh / a.kv_heads;
    const Request rq = request_of(a, b);
    if (rq.status != SV_ROW_OK) return;
    const Span sp = span_of(a, rq);
    if (PASS == 2 ? a.status[b] != SV_ROW_OK : pages_missing(a, sp, b)) return;
    const int64_t row = (int64_t)bh * a.ld_w;
    for (int i = share * 64 * WAVES + threadIdx.x; i < sp.tile0 * TILE; i += a.gap_blocks * 64 * WAVES)
      if (i >= sp.early * TILE) a.out[row + i] = a.in ? a.in[row + i] : 0.f;
    return;
  }
  const int h = it % a.kv_heads;
  it /= a.kv_heads;
  const int b = it % a.batch, chunk = a.chunks - 1 - it / a.batch;
  const Request rq = request_of(a, b);
  if (rq.status != SV_ROW_OK || (PASS == 2 && a.status[b] != SV_ROW_OK)) return;
  const Span sp = span_of(a, rq);
  const int used = (sp.tiles + a.chunk_tiles - 1) / a.chunk_tiles;
  const int begin = chunk * a.chunk_tiles, end = min(sp.tiles, begin + a.chunk_tiles);
  if (begin >= end) return;
  const int R = rq.count * a.group;
  const float c = a.scale * LOG2E;
  const uint8_t* pool = a.pages + (int64_t)h * a.unit;
  f32x2* const stats = (f32x2*)a.stats + ((int64_t)b * a.kv_heads + h) * a.chunks * a.max_rows;
  typename A::Pages id;
  const bool bad = id.ask(a, sp, a.table + (int64_t)b * a.ld_table, begin, end);
  const int mine = (end - begin - wave + WAVES - 1) / WAVES;  // the wave's tiles
  KTile<D> t[DEPTH];
  // the position of row r (fp32 divides these right: rows are below 2^16)
  auto position = [&](int r) { return rq.ctx + (int)(((float)min(r, R - 1) + 0.5f) * a.inv_group); };
  auto masked = [&](int base) {
    return base + TILE - 1 > rq.ctx ||
           (a.window > 0 && base <= rq.ctx + rq.rows - 1 - a.window && base + TILE > a.sinks);
  };
  // use(k-th tile of the wave, its codes) for all of them; DEPTH are on their way at any time,
  // behind the last ones the first again, for the next round.
  int ahead = 0;
  bool primed = false;
  auto ask = [&](KTile<D>& to) {
    A::fetch(a, to, pool, id, sp, begin + wave + ahead * WAVES);
    ahead = ahead + 1 < mine ? ahead + 1 : 0;
  };
  auto each_tile = [&](auto&& use) {
    if (mine <= 0) return;
    if (!primed) {
      ahead = 0;
#pragma unroll
      for (int k = 0; k < DEPTH; ++k) ask(t[k]);
    }
    for (int i = 0; i < mine; i += DEPTH) {
#pragma unroll
      for (int k = 0; k < DEPTH; ++k) {
        if (i + k < mine) use(i + k, t[k]);
        ask(t[k]);
      }
    }
    primed = mine % DEPTH == 0;               // (else the next round starts in another buffer)
  };

#pragma unroll
  for (int pass = 1; pass <= 2; ++pass) {
    if (!(PASS & pass)) continue;
    if (PASS == 3 && pass == 2) {             // a page id out of range: the request is left alone
      if (threadIdx.x == 0) any_bad = 0;
      __syncthreads();
      if (bad && lane == 0) any_bad = 1;
      __syncthreads();
      if (any_bad) return;
    }
    for (int g0 = 0; g0 < max(R, 1); g0 += a.group_rows) {
      const int rows = min(a.group_rows, R - g0), blocks = (rows + ROWS - 1) / ROWS;
      if (!(PASS == 3 && pass == 2 && R <= a.group_rows)) {
        __syncthreads();                      // (every wave is done with the rows before)
        A::put_q(a, q, rq, h, g0, blocks * MT, R, wave, WAVES);
        if (pass == 2)                        // the rows' maxima and sums over all chunks
          for (int i = threadIdx.x >> 3; i < blocks * ROWS; i += 8 * WAVES) {     // 8 lanes each
            float nm = -FAR, sum = 0.f;
            const f32x2* from = stats + g0 + min(i, rows - 1);
            for (int k = lane & 7; k < used; k += 32) {
              f32x2 y[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) y[u] = from[(int64_t)min(k + 8 * u, used - 1) * a.max_rows];
#pragma unroll
              for (int u = 0; u < 4; ++u)
                if (k + 8 * u < used) join(nm, sum, y[u][0], y[u][1]);
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) join(nm, sum, __shfl_xor(nm, d), __shfl_xor(sum, d));
            if ((lane & 7) == 0)              // (what is past the last row repeats it, and adds 0)
              fin[i] = f32x2{nm, i < rows && sum > 0.f && sum < INFINITY ? 1.f / sum : 0.f};
          }
        __syncthreads();
      }
      if (pass == 1) {
        if (mine <= 0)                        // (a wave without tiles leaves what counts nothing)
          for (int i = lane; i < rows; i += 64) part[wave * a.group_rows + i] = f32x2{-FAR, 0.f};
        for (int rb = 0; rb < blocks; ++rb) {
          if (mine <= 0) break;
          float m[MT], mc[MT], l[MT];
          int pos[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            pos[mt] = position(g0 + rb * ROWS + mt * 16 + n);
            m[mt] = -INFINITY;
            mc[mt] = -FAR;
            l[mt] = 0.f;
          }
          each_tile([&](int k, const KTile<D>& kt) {
            f32x4 s[2][MT];
            const int base = base_of(sp, begin + wave + k * WAVES);
            A::template scores<false>(a, kt, ONE ? q : q + rb * A::Q_WORDS, s, base, masked(base),
                                      [&](int mt, int) { return pos[mt]; });
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              float mx = m[mt];
#pragma unroll
              for (int i = 0; i < 8; ++i) mx = fmaxf(mx, s[i >> 2][mt][i & 3]);
              if (__any(mx > m[mt])) {        // (per lane: its tokens of the row)
                const float nc = __builtin_amdgcn_fmed3f(mx * c, -FAR, FAR);
                l[mt] *= __builtin_amdgcn_exp2f(mc[mt] - nc);
                m[mt] = mx;
                mc[mt] = nc;
              }
              float sum = 0.f;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                sum += __builtin_amdgcn_exp2f(__builtin_fmaf(s[i >> 2][mt][i & 3], c, -mc[mt]));
              l[mt] += sum;
            }
          });
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {   // join the row's four lanes
#pragma unroll
            for (int d = 16; d < 64; d <<= 1)
              join(mc[mt], l[mt], __shfl_xor(mc[mt], d), __shfl_xor(l[mt], d));
            if (g == 0) part[wave * a.group_rows + rb * ROWS + mt * 16 + n] = f32x2{mc[mt], l[mt]};
          }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < blocks * ROWS; i += 64 * WAVES) {    // then the waves
          float nm = -FAR, sum = 0.f;
#pragma unroll
          for (int k = 0; k < WAVES; ++k) {
            const f32x2 y = part[k * a.group_rows + min(i, rows - 1)];
            join(nm, sum, y[0], y[1]);
          }
          if (PASS == 3 && R <= a.group_rows)
            fin[i] = f32x2{nm, i < rows && sum > 0.f && sum < INFINITY ? 1.f / sum : 0.f};
          else if (i < rows)
            stats[(int64_t)chunk * a.max_rows + g0 + i] = f32x2{nm, sum};
        }
        if constexpr (PASS == 3) __syncthreads();
      } else {
        bool none = false;                    // some rows add nothing
        for (int i = lane; i < rows; i += 64) none |= fin[i][1] == 0.f;
        none = __any(none);
        f32x4 mc[MT], inv[MT];
        auto state = [&](int rb) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              const f32x4 y = *(const f32x4*)&fin[rb * ROWS + mt * 16 + 4 * g + i];
              mc[mt][i] = y[0];
              inv[mt][i] = y[1];
              mc[mt][i + 1] = y[2];
              inv[mt][i + 1] = y[3];
            }
        };
        if (ONE) state(0);
        each_tile([&](int k, const KTile<D>& kt) {
          const int at = wave + k * WAVES, base = base_of(sp, begin + at);
          const bool hide = masked(base);
          float w[2] = {};                    // of tokens n and 16 + n, over the lane's rows
          for (int rb = 0; rb < blocks; ++rb) {
            if (!ONE) state(rb);
            f32x4 s[2][MT];
            A::template scores<true>(
                a, kt, ONE ? q : q + rb * A::Q_WORDS, s, base, hide,
                [&](int mt, int i) { return position(g0 + rb * ROWS + mt * 16 + 4 * g + i); });
            if (none) {
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (inv[mt][i] == 0.f) s[0][mt][i] = s[1][mt][i] = -INFINITY;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
                  w[hf] = __builtin_fmaf(
                      __builtin_amdgcn_exp2f(__builtin_fmaf(s[hf][mt][i], c, -mc[mt][i])), inv[mt][i], w[hf]);
            if (ONE) break;
          }
          // over the lanes of a token: half of the tile each, then both lanes of a half
          const bool upper = g & 2;
          float y = (upper ? w[1] : w[0]) + __shfl_xor(upper ? w[0] : w[1], 32);
          y += __shfl_xor(y, 16);
          if (!(g & 1)) acc[at * TILE + 8 * g + n] = y;
        });
        __syncthreads();
        const int64_t row = ((int64_t)b * a.kv_heads + h) * a.ld_w;
        for (int i = threadIdx.x; i < (end - begin) * TILE; i += 64 * WAVES) {
          const int tok = base_of(sp, begin + i / TILE) + i % TILE;
          if (tok >= sp.n) continue;
          const float* before = g0 ? a.out : tok < rq.ctx ? a.in : nullptr;
          a.out[row + tok] = (before ? before[row + tok] : 0.f) + acc[i];
        }
      }
    }
  }
}

struct Plan {
  int mt, chunks, chunk_tiles, max_rows, group_rows;
  bool one;
  size_t bytes;
};

static bool plan_of(int dtype, int batch, int max_k, int heads, int kv_heads, int d, int max_context,
                    int window, int sinks, Plan& p) {
  const int64_t R = (int64_t)(max_k + 1) * (heads / kv_heads);
  const int nt = dtype == SV_F32 ? 3 : 1;
  p.mt = R <= 16 ? 1 : R <= 32 || (nt == 3 && d == 256) ? 2 : 4;
  p.one = R <= 32;
  p.max_rows = (int)R;
  // queries and statistics of a group of rows take at most 55 KiB of LDS, the weights of 64
  // tiles 8; the groups are even
  const int rows = 16 * p.mt, row_bytes = d * 2 * nt + (waves_of(true) + 1) * 8;
  const int64_t most = (65536 - 9216) / row_bytes / rows * rows, groups = (R + most - 1) / most;
  p.group_rows = (int)(((R + groups - 1) / groups + rows - 1) / rows * rows);
  int64_t tokens = max_context;
  if (window > 0) {
    const int64_t seen = (int64_t)window + max_k + 1 + sinks + 3 * TILE;
    if (seen < tokens) tokens = seen;
  }
  const int64_t tiles = (tokens + TILE - 1) / TILE, wide = (int64_t)batch * kv_heads;
  // one launch where every request has at most four tiles per wave, else chunks of 64 tiles
  // (whose pages a wave looks up at once), halved down to 256 tokens while there are less than
  // two workgroups per compute unit, four where fp32 rows make a tile three products (32
  // requests of 7 rows over 500 to 8,000 positions 44 us against 60; 8 requests of bf16 rows
  // over 500 to 16,000 took 41 with four, 36 with two)
  int64_t ct = SUB;
  if (tiles <= 4 * waves_of(true)) ct = 4 * waves_of(true);
  else
    while (ct > 8 && wide * ((tiles + ct - 1) / ct) < (nt == 3 ? 1024 : 512)) ct /= 2;
  p.chunks = (int)((tiles + ct - 1) / ct);
  p.chunk_tiles = (int)ct;
  if (wide * p.chunks >= (1ll << 23)) return false;
  p.bytes = (size_t)(wide * p.chunks * R) * 2 * sizeof(float) + 16;
  return true;
}

static bool sizes_ok(int dtype, int batch, int max_k, int heads, int kv_heads, int d, int max_context,
                     int window, int sinks) {
  return (dtype == SV_F32 || dtype == SV_BF16) && batch >= 1 && batch <= MAX_BATCH && max_k >= 0 &&
         max_k <= 63 && kv_heads >= 1 && heads >= kv_heads && heads % kv_heads == 0 && heads <= 1024 &&
         dim_ok(d) && max_context >= 1 && max_context <= (1 << 30) && window >= 0 &&
         window <= (1 << 30) && sinks >= 0 && sinks <= (1 << 30);
}

template <int D, int MT, bool ONE, typename T>
static int launch(const WeightArgs& a, const Plan& p, hipStream_t s) {
  const int items = a.batch * a.kv_heads * p.chunks, gaps = a.gap_blocks * a.batch * a.kv_heads;
  const int waves = waves_of(p.chunks == 1), statuses = (a.batch + waves - 1) / waves;
  const size_t queries = (size_t)p.group_rows * D * 2 * Weights<D, MT, T>::NT, stat = p.group_rows * 8;
  if (p.chunks == 1) {
    hipLaunchKernelGGL((k_weights<D, MT, ONE, 3, T>), dim3(statuses + items + gaps), dim3(64 * waves),
                       queries + (waves + 1) * stat, s, a);
    return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_LAUNCH;
  }
  hipLaunchKernelGGL((k_weights<D, MT, ONE, 1, T>), dim3(statuses + items), dim3(64 * waves),
                     queries + waves * stat, s, a);
  if (hipGetLastError() != hipSuccess) return SV_ERR_LAUNCH;
  hipLaunchKernelGGL((k_weights<D, MT, ONE, 2, T>), dim3(items + gaps), dim3(64 * waves),
                     queries + stat, s, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_LAUNCH;
}

// -------------------------------------------------------------------- evict
//
// Per layer, request and KV head a workgroup finds the weight of the last position that
// stays (a radix select over order-preserving keys), lists what stays, and moves it forward
// in order and in place, a slot per thread: slot i gets a position p >= i, so that where a
// step's positions are all read before its slots are written, no write reaches what a later
// step reads.  A second launch sets tables, counts and lengths, once all of them are done.
//
// What bounds it: the select (three passes over LDS counters, 22 us) and the list (10), then
// the moves, near HBM's rate: a token's V codes lie in 16 pieces 32 bytes apart (the layout in
// which attention reads them), so that lines of tokens that go are read too.  64 requests of
// 900 to 4,096 positions cut to 1,024, 2 layers: 111 us, 244 MB read and 132 written.  One
// workgroup per compute unit (256 of 32,768 positions): 133 us, 294 and 109 MB.

struct EvictArgs {
  const int32_t* budgets;
  int batch, sinks, recent;
  float* weights;
  int64_t ld_w;
  int kv_heads, page, page_log2, unit;
  int32_t* seq_lens;
  int32_t* table;
  int64_t ld_table;
  int32_t* refs;
  int64_t num_pages;
  uint8_t* pages;
  int64_t layer_bytes;
  int32_t* evicted;
  int32_t* status;
};

// Larger weights have larger keys, NaN the smallest; 0 and -0 are the same.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0;
  const uint32_t u = __builtin_bit_cast(uint32_t, w + 0.f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// A request's SV_ROW_*; n > m > 0 only where something is to be done.  All threads of the
// workgroup take part.
__device__ __forceinline__ int evict_status(const EvictArgs& a, int b, int& n, int& m) {
  n = a.seq_lens[b];
  m = a.budgets[b];
  if (n < 0 || n > a.ld_w || ((int64_t)n + a.page - 1) >> a.page_log2 > a.ld_table) {
    m = n = 0;
    return SV_ROW_BAD_PARAM;
  }
  if (m <= 0 || n <= m) {
    m = n = 0;
    return SV_ROW_OK;
  }
  if ((int64_t)a.sinks + a.recent > m) {
    m = n = 0;
    return SV_ROW_BAD_PARAM;
  }
  const int32_t* tab = a.table + (int64_t)b * a.ld_table;
  const int held = (n + a.page - 1) >> a.page_log2, kept = (m + a.page - 1) >> a.page_log2;
  bool bad = false;                           // outside the pool, or written and not its own
  for (int s = threadIdx.x; s < held; s += blockDim.x) {
    const uint32_t id = (uint32_t)tab[s];
    if (id >= (uint64_t)a.num_pages) bad = true;
    else if (s < kept && a.refs[id] != 1) bad = true;
  }
  if (!__syncthreads_or(bad)) return SV_ROW_OK;
  m = n = 0;
  return SV_ROW_BAD_PAGE;
}

// A token's V codes of a 16th of the dims.
template <int D> struct Piece { typedef uint32_t T; };
template <> struct Piece<64> { typedef uint16_t T; };
template <> struct Piece<256> { typedef u32x2 T; };

// A position's codes and scales: K in one piece, V in 16.
template <int D>
struct Token {
  u32x4 k[D / 32];
  typename Piece<D>::T v[16];
  uint8_t ks[D / 32], vs[D / 32];
  __device__ __forceinline__ void load(const uint8_t* u, int t, int P) {
    const uint8_t* pv = u + off_v(P, D) + (t >> 3) * (4 * D) + (t & 7) * (D / 32);
    const uint8_t* e = u + off_ks(P, D) + (t >> 3) * (D / 4) + (t & 7);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) k[i] = *(const u32x4*)(u + t * (D / 2) + 16 * i);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = *(const typename Piece<D>::T*)(pv + i * (D / 4));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      ks[i] = e[i * 8];
      vs[i] = e[P * (D / 32) + i * 8];
    }
  }
  __device__ __forceinline__ void store(uint8_t* u, int t, int P) const {
    uint8_t* pv = u + off_v(P, D) + (t >> 3) * (4 * D) + (t & 7) * (D / 32);
    uint8_t* e = u + off_ks(P, D) + (t >> 3) * (D / 4) + (t & 7);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) *(u32x4*)(u + t * (D / 2) + 16 * i) = k[i];
#pragma unroll
    for (int i = 0; i < 16; ++i) *(typename Piece<D>::T*)(pv + i * (D / 4)) = v[i];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      e[i * 8] = ks[i];
      e[P * (D / 32) + i * 8] = vs[i];
    }
  }
};

// THREADS threads; the weights of KEEP * THREADS positions stay in registers, those past them
// are read again at every use.
template <int D, int THREADS, int KEEP>
__global__ __launch_bounds__(THREADS, THREADS == 256 && D < 256 ? 5 : 1) void k_evict(EvictArgs a) {
  constexpr int BINS = 2048, WAVES = THREADS / 64, PER = BINS / THREADS;
  constexpr int LIST = 4 * THREADS < 4096 ? 2048 : 4096;      // positions that stay, listed at a time
  __shared__ int hist[BINS];
  __shared__ int wsum[WAVES], picked[2], wgt[WAVES], weq[WAVES];
  __shared__ int list[LIST];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = blockIdx.x % a.kv_heads, b = blockIdx.x / a.kv_heads % a.batch;
  const int layer = blockIdx.x / a.kv_heads / a.batch;
  int n, m;
  const int st = evict_status(a, b, n, m);
  if (layer == 0 && h == 0 && tid == 0) a.status[b] = st;
  if (m == 0) return;
  float* const w = a.weights + (int64_t)blockIdx.x * a.ld_w;
  const int lo = a.sinks, hi = n - a.recent;  // positions that are chosen among
  const int room = m - a.sinks - a.recent;    // how many of them stay
  // a wave has a stretch of the positions, in steps of 64
  const int steps = (n + THREADS - 1) / THREADS, from = wave * steps * 64;
  // (0 for positions that are not chosen among, and for NaN)
  auto key_at = [&](int i) {
    const int p = from + i * 64 + lane;
    return p >= lo && p < hi ? key_of(w[p]) : 0u;
  };
  uint32_t key[KEEP];
#pragma unroll
  for (int i = 0; i < KEEP; ++i) key[i] = i < steps ? key_at(i) : 0u;
  // the steps whose position is chosen among, and those whose position stays anyway
  uint32_t among = 0, always = 0;
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    const int p = from + i * 64 + lane;
    among |= (uint32_t)(i < steps && p >= lo && p < hi) << i;
    always |= (uint32_t)(i < steps && p < n && (p < lo || p >= hi)) << i;
  }
  auto is_among = [&](int i) {
    const int p = from + i * 64 + lane;
    return i < KEEP ? (bool)(among >> i & 1) : p >= lo && p < hi;
  };
  // each(f): f(step, key) for the wave's positions, in order
  auto each = [&](auto&& f) {
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
      if (i < steps) f(i, key[i]);
    for (int i = KEEP; i < steps; ++i) f(i, key_at(i));
  };

  uint32_t last = 0xffffffffu;                // the key of the last that stays (no weight has this one)
  int ties = 0;                               // of those with just this key, the first so many stay
  if (room > 0) {
    ties = room;
    last = 0;
    uint32_t mask = 0;
    for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift == 10 ? 0 : -1) {
      const int bits = shift == 0 ? 10 : 11;
      for (int i = tid; i < BINS; i += THREADS) hist[i] = 0;
      __syncthreads();
      each([&](int i, uint32_t k) {
        if (is_among(i) && (k & mask) == last) atomicAdd(&hist[k >> shift & ((1 << bits) - 1)], 1);
      });
      __syncthreads();
      // digits from the top: thread t takes the PER bins below BINS - PER t
      int c[PER], sum = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        c[i] = hist[BINS - 1 - (tid * PER + i)];
        sum += c[i];
      }
      int upto = sum;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(upto, d);
        if (lane >= d) upto += y;
      }
      if (lane == 63) wsum[wave] = upto;
      __syncthreads();
      for (int k = 0; k < wave; ++k) upto += wsum[k];
      int before = upto - sum;                // in larger digits
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (before < ties && ties <= before + c[i]) {
          picked[0] = BINS - 1 - (tid * PER + i);
          picked[1] = before;
        }
        before += c[i];
      }
      __syncthreads();
      last |= (uint32_t)picked[0] << shift;
      mask |= ((1u << bits) - 1) << shift;
      ties -= picked[1];
    }
  }
  // what stays whatever the ties, and the ties
  auto sure_of = [&](int i, uint32_t k) {
    const int p = from + i * 64 + lane;
    const bool stays = i < KEEP ? (bool)(always >> i & 1) : p < n && (p < lo || p >= hi);
    return stays || (is_among(i) && k > last);
  };
  auto tie_of = [&](int i, uint32_t k) {
    return room > 0 && is_among(i) && k == last;
  };
  int gt = 0, eq = 0;
  each([&](int i, uint32_t k) {
    gt += __popcll(__ballot(sure_of(i, k)));
    eq += __popcll(__ballot(tie_of(i, k)));
  });
  if (lane == 0) {
    wgt[wave] = gt;
    weq[wave] = eq;
  }
  __syncthreads();
  int slot0 = 0, tie0 = 0;                    // of the waves before
  for (int v = 0; v < wave; ++v) {
    slot0 += wgt[v] + max(0, min(ties - tie0, weq[v]));
    tie0 += weq[v];
  }

  // move: slot i gets position list[i], LIST slots at a time
  const int32_t* tab = a.table + (int64_t)b * a.ld_table;
  uint8_t* const pool = a.pages + layer * a.layer_bytes + (int64_t)h * a.unit;
  const int64_t page_bytes = (int64_t)a.unit * a.kv_heads;
  const int P = a.page;
  // A list ends within a wave's step as a rule: the wave goes on from there, with the step's
  // ballots as they were.  Weights are never read again where the moves have changed them: in
  // steps after slot s0 every position is s0 or more.
  int slot = slot0, tied = tie0, next = 0;    // before the step that the wave goes on with
  uint64_t bs = 0, bt = 0;
  bool held = false;                          // its ballots are known
  for (int s0 = 0; s0 < m; s0 += LIST) {
    const int s1 = min(m, s0 + LIST);
    __syncthreads();                          // (the list before is used up)
    auto put = [&](int i, auto&& key_of_step) {
      if (i != next || slot >= s1) return;
      if (!held) {
        const uint32_t k = key_of_step(i);
        bs = __ballot(sure_of(i, k));
        bt = __ballot(tie_of(i, k));
      }
      const uint64_t below = (1ull << lane) - 1;
      const int my_ties = min(max(ties - tied, 0), (int)__popcll(bt & below));
      const bool keep = (bs >> lane & 1) || ((bt >> lane & 1) && tied + (int)__popcll(bt & below) < ties);
      const int to = slot + __popcll(bs & below) + my_ties;
      if (keep && to >= s0 && to < s1) list[to - s0] = from + i * 64 + lane;
      const int after = slot + __popcll(bs) + min(max(ties - tied, 0), (int)__popcll(bt));
      held = after > s1;
      if (held) return;
      slot = after;
      tied += __popcll(bt);
      next = i + 1;
    };
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
      if (i < steps) put(i, [&](int x) { return key[x]; });
    for (int i = max(KEEP, next); i < steps && i == next && slot < s1; ++i) put(i, key_at);
    __syncthreads();
    for (int i0 = s0; i0 < s1; i0 += THREADS) {
      const int to = i0 + tid, p = to < s1 ? list[to - s0] : to;
      const bool move = p != to;
      Token<D> y;
      float x;
      if (move) {
        x = w[p];
        y.load(pool + tab[p >> a.page_log2] * page_bytes, p & (P - 1), P);
      }
      __syncthreads();                        // (all are read before one is written)
      if (move) {
        w[to] = x;
        y.store(pool + tab[to >> a.page_log2] * page_bytes, to & (P - 1), P);
      }
    }
  }
  __syncthreads();
  for (int p = m + tid; p < n; p += THREADS) w[p] = 0.f;
}

// Tables, counts and lengths of the requests that k_evict cut: a workgroup each.
__global__ __launch_bounds__(256) void k_evict_tables(EvictArgs a) {
  const int b = blockIdx.x;
  const int n = a.seq_lens[b], m = a.budgets[b];
  if (a.status[b] != SV_ROW_OK || m <= 0 || n <= m) return;
  int32_t* const tab = a.table + (int64_t)b * a.ld_table;
  const int held = (n + a.page - 1) >> a.page_log2, kept = (m + a.page - 1) >> a.page_log2;
  for (int s = kept + threadIdx.x; s < held; s += 256) {
    atomicAdd(&a.refs[tab[s]], -1);
    tab[s] = -1;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    a.seq_lens[b] = m;
    if (a.evicted) a.evicted[b] += n - m;
  }
}

}  // namespace budget
}  // namespace svk

using namespace svk;

extern "C" {

size_t spec_kv_weights_workspace_bytes(int dtype, int batch, int max_k, int heads, int kv_heads,
                                       int head_dim, int max_context, int window, int sinks) {
  budget::Plan p;
  if (!budget::sizes_ok(dtype, batch, max_k, heads, kv_heads, head_dim, max_context, window, sinks) ||
      !budget::plan_of(dtype, batch, max_k, heads, kv_heads, head_dim, max_context, window, sinks, p))
    return 0;
  return p.bytes;
}

int spec_kv_attention_weights(const void* q, int64_t ld_q, int dtype, const int32_t* cu_seqlens,
                              const int32_t* context_lens, const int32_t* row_counts, int batch,
                              int total_rows, int max_k, int heads, int kv_heads, int head_dim,
                              const void* pages, int64_t num_pages, int page_size,
                              const int32_t* page_table, int64_t ld_table, int max_context,
                              float scale, int window, int sinks, const float* weights_in,
                              float* weights_out, int64_t ld_weights, int32_t* status,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !cu_seqlens || !context_lens || !pages || !page_table || !weights_out || !status)
    return SV_ERR_NULL;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  budget::Plan p;
  if (!budget::sizes_ok(dtype, batch, max_k, heads, kv_heads, head_dim, max_context, window, sinks) ||
      total_rows < 1 || !page_ok(page_size) || num_pages < 1 || num_pages > 0x7fffffff ||
      ld_table < 1 || ld_table > (1 << 30) / page_size || ld_q < (int64_t)heads * head_dim ||
      ld_weights < max_context || !(scale > 0.f) || !(scale <= 2.0e38f) || !aligned16(pages) ||
      !budget::plan_of(dtype, batch, max_k, heads, kv_heads, head_dim, max_context, window, sinks, p))
    return SV_ERR_SHAPE;
  if (weights_in && weights_in != weights_out) {
    const uintptr_t in = (uintptr_t)weights_in, out = (uintptr_t)weights_out;
    const size_t bytes = (size_t)batch * kv_heads * ld_weights * sizeof(float);
    if ((in < out ? out - in : in - out) < bytes) return SV_ERR_SHAPE;
  }
  if (!workspace || !aligned16(workspace)) return SV_ERR_NULL;
  if (p.bytes > workspace_bytes) return SV_ERR_WORKSPACE;
  budget::WeightArgs a;
  a.q = q;
  a.ld_q = ld_q;
  a.cu = cu_seqlens;
  a.ctx = context_lens;
  a.counts = row_counts;
  a.batch = batch;
  a.total_rows = total_rows;
  a.max_k = max_k;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.group = heads / kv_heads;
  a.inv_group = 1.f / (float)a.group;
  a.pages = (const uint8_t*)pages;
  a.num_pages = num_pages;
  a.page = page_size;
  a.page_log2 = __builtin_ctz((unsigned)page_size);
  a.unit = (int)unit_bytes(page_size, head_dim);
  a.table = page_table;
  a.ld_table = ld_table;
  a.max_context = max_context;
  a.scale = scale;
  a.window = window;
  a.sinks = sinks;
  a.in = weights_in;
  a.out = weights_out;
  a.ld_w = ld_weights;
  a.status = status;
  a.chunks = p.chunks;
  a.chunk_tiles = p.chunk_tiles;
  a.max_rows = p.max_rows;
  a.group_rows = p.group_rows;
  a.stats = (float*)workspace;
  a.gap_blocks = 0;
  if (window > 0 && weights_in != weights_out) {
    const int64_t more = (max_context + 8191) / 8192, most = (1 << 22) / (batch * kv_heads);
    a.gap_blocks = (int)(more < most ? more : most);
    if (a.gap_blocks < 1) a.gap_blocks = 1;
  }
  hipStream_t s = (hipStream_t)stream;
#define SVK_CASE(DD, MM, OO, TT) \
  if (head_dim == DD && p.mt == MM && p.one == OO) return budget::launch<DD, MM, OO, TT>(a, p, s)
#define SVK_CASES(DD, TT)          \
  SVK_CASE(DD, 1, true, TT);       \
  SVK_CASE(DD, 2, true, TT)
  if (dtype == SV_BF16) {
    SVK_CASES(64, __bf16);
    SVK_CASES(128, __bf16);
    SVK_CASES(256, __bf16);
    SVK_CASE(64, 4, false, __bf16);
    SVK_CASE(128, 4, false, __bf16);
    SVK_CASE(256, 4, false, __bf16);
  } else {
    SVK_CASES(64, float);
    SVK_CASES(128, float);
    SVK_CASES(256, float);
    SVK_CASE(64, 4, false, float);
    SVK_CASE(128, 4, false, float);
    SVK_CASE(256, 2, false, float);
  }
#undef SVK_CASES
#undef SVK_CASE
  return SV_ERR_SHAPE;
}

int spec_kv_evict(const int32_t* budgets, int batch, int sinks, int recent, float* weights,
                  int64_t ld_weights, int kv_heads, int head_dim, int page_size, int32_t* seq_lens,
                  int32_t* page_table, int64_t ld_table, int32_t* ref_counts, int64_t num_pages,
                  void* pages, int layers, int64_t layer_bytes, int32_t* evicted, int32_t* status,
                  void* stream) {
  if (!budgets || !weights || !seq_lens || !page_table || !ref_counts || !pages || !status)
    return SV_ERR_NULL;
  if (batch < 1 || batch > MAX_BATCH || sinks < 0 || sinks > (1 << 30) || recent < 0 ||
      recent > (1 << 30) || ld_weights < 1 || kv_heads < 1 || kv_heads > 1024 || !dim_ok(head_dim) ||
      !page_ok(page_size) || ld_table < 1 || ld_table > (1 << 30) / page_size || num_pages < 1 ||
      num_pages > (1 << 24) || !aligned16(pages) || layers < 1 || layers > 65535 ||
      layer_bytes % 16 != 0 || (int64_t)layers * batch * kv_heads >= (1 << 22) ||
      (layers > 1 && layer_bytes < num_pages * kv_heads * unit_bytes(page_size, head_dim)))
    return SV_ERR_SHAPE;
  budget::EvictArgs a;
  a.budgets = budgets;
  a.batch = batch;
  a.sinks = sinks;
  a.recent = recent;
  a.weights = weights;
  a.ld_w = ld_weights;
  a.kv_heads = kv_heads;
  a.page = page_size;
  a.page_log2 = __builtin_ctz((unsigned)page_size);
  a.unit = (int)unit_bytes(page_size, head_dim);
  a.seq_lens = seq_lens;
  a.table = page_table;
  a.ld_table = ld_table;
  a.refs = ref_counts;
  a.num_pages = num_pages;
  a.pages = (uint8_t*)pages;
  a.layer_bytes = layer_bytes;
  a.evicted = evicted;
  a.status = status;
  hipStream_t s = (hipStream_t)stream;
  const dim3 grid((uint32_t)(layers * batch * kv_heads));
  // 256 threads where they hold whole rows in registers or the workgroups are many, 1,024 for
  // long rows (us, with 256 and with 1,024: 512 rows of 900 to 4,096 positions 69 and 90, 8 of
  // 4,000 38 and 42, 1,024 of 16,000 444 and 490; 512 of 16,000 275 and 257, 64 of 8,000 78 and
  // 65, 256 of 8,000 to 32,768 242 and 143)
  const bool small = grid.x >= 1024 || ld_weights <= 16 * 256;
#define SVK_CASE(DD)                                                                              \
  if (head_dim == DD) {                                                                           \
    if (small) hipLaunchKernelGGL((budget::k_evict<DD, 256, 16>), grid, dim3(256), 0, s, a);      \
    else                                                                                          \
      hipLaunchKernelGGL((budget::k_evict<DD, 1024, DD == 256 ? 16 : 32>), grid, dim3(1024), 0,   \
                         s, a);                                                                   \
  }
  SVK_CASE(64)
  SVK_CASE(128)
  SVK_CASE(256)
#undef SVK_CASE
  if (hipGetLastError() != hipSuccess) return SV_ERR_LAUNCH;
  hipLaunchKernelGGL(budget::k_evict_tables, dim3(batch), dim3(256), 0, s, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_LAUNCH;
}

}  // extern "C"
