// kvattn.hip -- spec_kv_attention: the k+1 verify rows of each request over
// the 4-bit paged cache (include/specverify.h states the operator).
//
// For request b, row j (position c+j) and query head h over KV head h/G:
//   out = sum_t exp(scale q.k_t - m) v_t / sum_t exp(scale q.k_t - m)
// over the visible t, in one pass with a running maximum m and sum.
//
// One workgroup (2, 4 or 8 waves) takes one KV head, up to 16*MT of the
// R = (k+1)*G rows that share it, and one chunk of the context; its waves take
// the tiles of 32 tokens in turn and work alone until the end, where their
// partial results are joined through LDS.  A wave computes
//   S^T[token][row] = K Q^T   then   O^T[dim][row] += V^T P^T
// with v_mfma_f32_16x16x32_bf16.  With tokens as the rows of S^T, a lane holds
// the scores of ONE query row (its column), for 8 tokens (4 of each half of the
// tile) that are exactly the 8 contraction entries of its P^T operand: softmax
// statistics are per lane and the probabilities go from accumulator to operand
// without LDS or shuffles.  K and V come as e2m1 codes and are widened to bf16 by the
// hardware conversion, which applies the power-of-two block scale (exact).
//
// What bounds it: the vector instructions that widen the cache (half a conversion
// and, for V, half a byte permutation per value of a tile and row block) and make the
// softmax, and HBM reads (D*17/16 bytes per token and KV head), which do not overlap
// fully at two waves per SIMD.  64 requests over 512 to 16,384 positions (k=6, 32
// heads over 8 KV heads of D=128, 301 MB): 80 us, of these plan 5, this kernel 69
// (4.4 TB/s, vector units busy 52 % and matrix units 27 % of the time), join 7.  One
// user over 32,000 positions, k=0: 18 us, of these join 4.2; 64 requests over 4,000
// with 64 heads (R=56, two row blocks that both read and widen the cache): 124 us,
// 470 TFLOP/s.

#include "kv_common.h"

namespace svk {

constexpr int TILE = 32;          // tokens per wave step
constexpr float LOG2E = 1.44269504088896340736f;
// the running maximum is raised only when a score passes it by this much (in
// powers of two): until then weights stay below 2^8, which fp32 sums and bf16
// weights hold with the same relative precision
constexpr float RAISE = 8.0f;
// Weights are 2^(s c - mc), c = scale log2 e, with one rounding of the exponent; mc is
// the maximum m times c, rounded.  Everything is counted from mc (raises and joins
// too), so what mc is off by cancels in the division, but the largest weight is
// 2^(m c - mc): half a step of mc, 2^32 at most up to here.  mc is held within +-FAR: past
// it weights become infinite, or all 0, and their row NaN.
// (Weights 2^((s - m) c) would have no such end, at an instruction more per score: the
// windowed batch of 256 requests 61.3 us, with this 59.5, the verify batch 77.5 and 76.4.)
constexpr float FAR = 1073741824.0f;          // 2^30

struct AttnArgs {
  const void* q;
  int64_t ld_q;
  const int32_t* cu;
  const int32_t* ctx;
  int batch, total_rows, max_k, heads, kv_heads;
  int group;            // heads / kv_heads
  float inv_group;
  const uint8_t* pages;
  int64_t num_pages;
  int page, page_log2, unit;        // tokens of a page; bytes of a page's KV head
  const int32_t* table;
  int64_t ld_table;
  int max_context;
  float scale;
  int window, sinks;
  void* out;
  int64_t ld_out;
  int32_t* status;
  float* part;          // chunk partials: [item][rows][D], then [item][rows][2] (max, sum)
  int chunks, chunk_tiles, row_blocks, block_rows;   // chunks of a request at most
  struct Item* plan;    // [1 + items], the first holds how many there are; or NULL
};

// The tiles a request reads: tokens that some row sees, in steps of 32.
struct Span {
  int n;            // positions up to the last row's, exclusive
  int first;        // first position row 0's window shows
  int sink_tiles, tile0, tiles;
};

__device__ __forceinline__ Span span_of(int ctx, int rows, int window, int sinks) {
  Span s;
  s.n = ctx + rows;
  s.first = window > 0 ? max(0, ctx - window + 1) : 0;
  s.tile0 = s.first / TILE;
  s.sink_tiles = min((sinks + TILE - 1) / TILE, s.tile0);
  s.tiles = s.sink_tiles + (s.n - 1) / TILE - s.tile0 + 1;
  return s;
}

// Tiles of a chunk of a request: the call's, or more where the request would have more
// chunks than the call has places for.
__device__ __forceinline__ int chunk_of(const AttnArgs& a, int tiles) {
  return tiles <= a.chunks * a.chunk_tiles ? a.chunk_tiles : (tiles + a.chunks - 1) / a.chunks;
}

// A request's numbers and its SV_ROW_* by them alone (pages are checked where
// read).  One wave; its loads go out together with those of the offsets' check.
__device__ __forceinline__ int request_status(const AttnArgs& a, int b, int& row0, int& rows,
                                              int& ctx) {
  const int c0 = a.cu[b], c1 = a.cu[b + 1], cx = a.ctx[b];
  const int broken = first_broken(a.cu, a.batch, a.total_rows);
  row0 = rows = ctx = 0;
  if (b >= broken) return SV_ROW_BAD_K;
  row0 = c0;
  rows = c1 - c0;
  if (rows < 1 || rows > a.max_k + 1) return SV_ROW_BAD_K;
  ctx = cx;
  if (ctx < 0 || (int64_t)ctx + rows > a.max_context) return SV_ROW_BAD_PARAM;
  return SV_ROW_OK;
}

__device__ __forceinline__ bool page_needed(const Span& s, int slot, int page_log2, int sinks) {
  const int t0 = slot << page_log2, t1 = t0 + (1 << page_log2);
  return t0 < s.n && (t1 > s.first || t0 < sinks);
}

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__bf16>(__bf16 x) { return (float)x; }

// Combine over the four lanes that hold one query row (lanes l, l^16, l^32, l^48).
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
// A scale byte as the float 2^(byte-127).
__device__ __forceinline__ float scale_of(uint32_t word, int byte) {
  return __builtin_bit_cast(float, ((word >> (8 * byte)) & 255u) << 23);
}
template <int BYTE>
__device__ __forceinline__ uint32_t widen(uint32_t word, float scale) {
  return __builtin_bit_cast(uint32_t,
                            __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, BYTE));
}

// A lane's operands of a tile, for each half of 16 tokens.
template <int D>
struct Tile {
  uint32_t k[2][D / 32];              // token n, D/4 dims
  uint32_t ks[2][(D + 127) / 128];    // its scale bytes, per block of the lane's dims
  uint32_t v[D / 16];                 // tokens 4g .. 4g+3 of each half, D/16 dims
  uint32_t vs[2];                     // their scale bytes
};

// A workgroup's share, the same for all its threads.
struct Share {
  Span sp;
  int row0, ctx, rows, R;       // query rows: first in the call, position, count, times G
  int rb, tbegin, tend;         // row block, tiles
  float c;                      // scale log2 e
  const uint8_t* pool;          // the KV head's unit of page 0
  uint32_t page_bytes;
};

template <int D, int MT, typename T>
struct Attn {
  static constexpr int STEPS = D / 32;           // contraction steps of K Q^T
  static constexpr int FR = D / 16;              // output fragments of 16 dims
  static constexpr int KB = (D + 127) / 128;     // scale blocks of a lane's K dims
  // fp32 queries and weights are split into three bf16 terms (3 x 8 bits hold
  // fp32's 24): products with the exact bf16 K and V then lose nothing.  The weights of
  // bf16 rows are rounded to one term, and the sum they are divided by is that of the
  // rounded ones, so the roundings are independent errors of at most 2^-8 of each weight
  // that average out over the tokens like the values do: 0.0023 of the result's norm from
  // 64 bits, of which the result's own rounding to bf16 is 0.0017.  Two terms leave only
  // that 0.0017, for 86 us instead of 75 in the verify batch, 72 instead of 59 in the
  // windowed one and 63 instead of 54 at D=256; the caller who needs more bits than the
  // result's has fp32 rows.
  static constexpr int NT = sizeof(T) == 4 ? 3 : 1;

  f32x4 o[MT][FR];
  f32x4 l[MT];            // sums of the weights: a row of ones among the products (4 equal)
  // running max m of the raw scores: m, mc = m scale log2 e, rounded (-FAR before the
  // first visible score), and what a score has to pass to raise it
  float m[MT], mc[MT], over[MT];
  // rows that saw a block stored as NaN.  V: bit 4 mt + r, dims g*D/4 + r*D/16 ...;
  // K: bit 16 + mt, all dims
  uint32_t poison = 0;

  static __device__ __forceinline__ void split(float x, __bf16* t) {
    float r = x;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      t[i] = (__bf16)r;
      r -= (float)t[i];
    }
  }

  // Row r of a request's R: verify row r / G, query head r % G of the KV head's G
  // (fp32 divides these right: r < 2^16).
  static __device__ __forceinline__ int row_of(const AttnArgs& a, int r) {
    return (int)(((float)r + 0.5f) * a.inv_group);
  }

  // The query rows' operands lie in LDS, [row tile][step][term][lane], for all waves of
  // the workgroup: in registers they would take the place of a tile on its way.
  static constexpr int Q_BYTES = MT * STEPS * NT * 64 * 16;
  // A wave's share of them: requested first, written once they are there.
  template <int WAVES>
  struct Raw {
    static constexpr int N = (MT * STEPS + WAVES - 1) / WAVES;
    T x[N][8];
    __device__ __forceinline__ void ask(const AttnArgs& a, const Share& w, int h, int wave) {
      const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int at = min(wave + i * WAVES, MT * STEPS - 1), mt = at / STEPS, s = at % STEPS;
        const int r = min((w.rb * MT + mt) * 16 + n, w.R - 1);
        const int j = row_of(a, r), hq = h * a.group + r - j * a.group;
        __builtin_memcpy(x[i], (const T*)a.q + (int64_t)(w.row0 + j) * a.ld_q +
                                   (uint32_t)(hq * D + g * (D / 4) + 8 * s), sizeof(x[i]));
      }
    }
    __device__ __forceinline__ void put(bf16x8* q, int wave) const {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int at = wave + i * WAVES;
        if (MT * STEPS % WAVES != 0 && at >= MT * STEPS) continue;
        bf16x8 y[NT];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          __bf16 t[NT];
          if constexpr (NT == 1) t[0] = x[i][k];
          else split(to_f32<T>(x[i][k]), t);
#pragma unroll
          for (int u = 0; u < NT; ++u) y[u][k] = t[u];
        }
#pragma unroll
        for (int u = 0; u < NT; ++u) q[(at * NT + u) * 64 + (threadIdx.x & 63)] = y[u];
      }
    }
  };
  __device__ __forceinline__ void init() {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt] = over[mt] = -INFINITY;
      mc[mt] = -FAR;
      l[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int f = 0; f < FR; ++f) o[mt][f] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }

  // Half hf of a tile: 16 tokens at token `tb` of a page's unit.  The unit is a
  // buffer resource with a scalar base, the token a scalar offset, and the lane's
  // offsets are the same in every tile: a load costs no vector arithmetic.
  struct Lane {
    uint32_t k, ks, v, vs;
  };
  static __device__ __forceinline__ Lane lane_offsets(int P) {
    const uint32_t lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    Lane o;
    o.k = n * (D / 2) + g * (D / 8);
    o.ks = off_ks(P, D) + (n >> 3) * (D / 4) + (g * (D / 4) / 32) * 8 + (n & 7);
    o.v = off_v(P, D) + (g >> 1) * (4 * D) + n * (D / 4) + (g & 1) * (D / 8);
    o.vs = off_vs(P, D) + (g >> 1) * (D / 4) + (n * D / 512) * 8 + (g & 1) * 4;
    return o;
  }
  static __device__ __forceinline__ void load(Tile<D>& t, int hf, const uint8_t* unit, int bytes,
                                              const Lane& at, int tb) {
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc((void*)unit, 0, bytes, 0x00020000);
    const int sk = tb * (D / 2), ss = tb * (D / 32);
    if constexpr (D == 64) {
      const u32x2 k = __builtin_amdgcn_raw_buffer_load_b64(r, at.k, sk, 0);
      t.k[hf][0] = k[0];
      t.k[hf][1] = k[1];
      const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(r, at.v, sk, 0);
      t.v[hf * 2] = v[0];
      t.v[hf * 2 + 1] = v[1];
    } else {
#pragma unroll
      for (int i = 0; i < D / 128; ++i) {
        const u32x4 k = __builtin_amdgcn_raw_buffer_load_b128(r, at.k + 16 * i, sk, 0);
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, at.v + 16 * i, sk, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          t.k[hf][4 * i + j] = k[j];
          t.v[hf * (D / 32) + 4 * i + j] = v[j];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < KB; ++i)
      t.ks[hf][i] = __builtin_amdgcn_raw_buffer_load_b8(r, at.ks + 8 * i, ss, 0);
    t.vs[hf] = __builtin_amdgcn_raw_buffer_load_b32(r, at.vs, ss, 0);
  }
  // Entry i of a lane's 8 tokens, relative to the tile.
  static __device__ __forceinline__ int token(int g, int i) {
    return 16 * (i >> 2) + 4 * g + (i & 3);
  }

  // One tile for the first M row tiles.  masked: some row does not see some token.
  template <int M>
  __device__ __forceinline__ void step(const AttnArgs& a, Tile<D>& t, bool masked, int base,
                                       const Share& w, const bf16x8* q) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    int ql = lane;
    asm volatile("" : "+v"(ql));              // (or the reads move out of the loop, into registers)
    auto sees = [&](int tok, int pos) {
      return tok <= pos && (a.window == 0 || tok > pos - a.window || tok < a.sinks);
    };
    if (masked) {
      // tokens that no row sees (past the end, or between sinks and window) may
      // hold anything: their V becomes finite, so that a weight of 0 keeps it out
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int tok = base + token(g, i);
        if (tok >= w.sp.n || (tok < w.sp.first && tok >= a.sinks)) {
          const int sh = 8 * (i & 3);
          t.vs[i >> 2] = (t.vs[i >> 2] & ~(255u << sh)) | (127u << sh);
        }
      }
    }
    float ksc[2][KB], vsc[8];
    uint32_t top = 0;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        ksc[hf][i] = __builtin_bit_cast(float, t.ks[hf][i] << 23);
        top = max(top, t.ks[hf][i] << 23);
      }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      vsc[i] = scale_of(t.vs[i >> 2], i & 3);
      top = max(top, __builtin_bit_cast(uint32_t, vsc[i]));
    }
    if (__any(top == 0x7f800000u)) {          // a scale of 255: a block stored as NaN
      nan_blocks<M>(a, t, base, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) vsc[i] = scale_of(t.vs[i >> 2], i & 3);
    }
    // scores: s[half][mt], lane: row n, tokens base + 16*half + 4g + r
    f32x4 s[2][M];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int mt = 0; mt < M; ++mt) s[hf][mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
      bf16x8 qt[M][NT];
#pragma unroll
      for (int mt = 0; mt < M; ++mt)
#pragma unroll
        for (int k = 0; k < NT; ++k) qt[mt][k] = q[((mt * STEPS + st) * NT + k) * 64 + ql];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float sc = ksc[hf][st / 4];
        const uint32_t x = t.k[hf][st];
        u32x4 kb;
        kb[0] = widen<0>(x, sc);
        kb[1] = widen<1>(x, sc);
        kb[2] = widen<2>(x, sc);
        kb[3] = widen<3>(x, sc);
        const bf16x8 ka = __builtin_bit_cast(bf16x8, kb);
#pragma unroll
        for (int mt = 0; mt < M; ++mt)
#pragma unroll
          for (int k = NT - 1; k >= 0; --k)
            s[hf][mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ka, qt[mt][k], s[hf][mt], 0, 0, 0);
      }
    }
    if (masked) {
#pragma unroll
      for (int mt = 0; mt < M; ++mt) {
        // (lanes past the last row repeat it, in what they see too: they take part in
        // raising the tile's maxima)
        const int pos = w.ctx + row_of(a, min((w.rb * MT + mt) * 16 + n, w.R - 1));
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!sees(base + token(g, i), pos)) s[i >> 2][mt][i & 3] = -INFINITY;
      }
    }
    bf16x8 p[M][NT];
#pragma unroll
    for (int mt = 0; mt < M; ++mt) {
      float mx = fmaxf(fmaxf(s[0][mt][0], s[0][mt][1]), s[0][mt][2]);
      mx = fmaxf(fmaxf(mx, s[0][mt][3]), s[1][mt][0]);
      mx = fmaxf(fmaxf(mx, s[1][mt][1]), s[1][mt][2]);
      mx = fmaxf(mx, s[1][mt][3]);
      // (a first visible score raises -inf; a row that has seen nothing stays there)
      if (__any(mx > over[mt])) {
        const float nm = fmaxf(m[mt], row_max(mx));
        const float nc = __builtin_amdgcn_fmed3f(nm * w.c, -FAR, FAR);
        const float f = __builtin_amdgcn_exp2f(mc[mt] - nc);
        l[mt] *= f;
#pragma unroll
        for (int k = 0; k < FR; ++k) o[mt][k] *= f;
        m[mt] = nm;
        mc[mt] = nc;
        // (finite for the smallest scales too: a row that has seen nothing stays at -inf,
        // so that its first visible score raises it)
        over[mt] = nm + __builtin_fminf(RAISE / w.c, 3.4e38f);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i >> 2][mt][i & 3], w.c, -mc[mt]));
        __bf16 x[NT];
        split(e, x);
#pragma unroll
        for (int k = 0; k < NT; ++k) p[mt][k][i] = x[k];
      }
    }
    {
      bf16x8 one;
#pragma unroll
      for (int i = 0; i < 8; ++i) one[i] = (__bf16)1.f;
#pragma unroll
      for (int mt = 0; mt < M; ++mt)
#pragma unroll
        for (int k = NT - 1; k >= 0; --k)
          l[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(one, p[mt][k], l[mt], 0, 0, 0);
    }
    // fragment pair c2: dims 2*c2 and 2*c2+1 of every lane's D/16
#pragma unroll
    for (int c2 = 0; c2 < FR / 2; ++c2) {
      uint32_t x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int byte = i * (D / 32) + c2;
        const uint32_t v = t.v[byte / 4];
        x[i] = byte % 4 == 0 ? widen<0>(v, vsc[i]) : byte % 4 == 1 ? widen<1>(v, vsc[i])
             : byte % 4 == 2 ? widen<2>(v, vsc[i]) : widen<3>(v, vsc[i]);
      }
      u32x4 lo, hi;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x05040100u);
        hi[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x07060302u);
      }
#pragma unroll
      for (int mt = 0; mt < M; ++mt)
#pragma unroll
        for (int k = NT - 1; k >= 0; --k) {
          o[mt][2 * c2] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, lo), p[mt][k], o[mt][2 * c2], 0, 0, 0);
          o[mt][2 * c2 + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, hi), p[mt][k], o[mt][2 * c2 + 1], 0, 0, 0);
        }
    }
  }

  // Blocks stored as NaN.  K: every row that sees the token is NaN.  V: such a row
  // gets NaN in the block's dims.  The others must not (0 * NaN), so `poison` keeps
  // who saw what and V is made finite for the products; the scores that a K block
  // spoils are those of rows that are NaN anyway or that the mask replaces.
  template <int M>
  __device__ __forceinline__ void nan_blocks(const AttnArgs& a, Tile<D>& t, int base,
                                             const Share& w) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    auto sees = [&](int tok, int mt) {
      const int pos = w.ctx + row_of(a, (w.rb * MT + mt) * 16 + n);
      return tok <= pos && (a.window == 0 || tok > pos - a.window || tok < a.sinks);
    };
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      bool odd = false;
#pragma unroll
      for (int i = 0; i < KB; ++i) odd |= t.ks[hf][i] == 255u;
      uint64_t b = __ballot(odd);             // bit 16 g + n: token n
      b |= b >> 32;
      b = (b | b >> 16) & 0xffffu;
      for (; b; b &= b - 1)
#pragma nounroll
        for (int mt = 0; mt < M; ++mt)
          if (sees(base + 16 * hf + __builtin_ctzll(b), mt)) poison |= 0x10000u << mt;
    }
#pragma nounroll
    for (int src = 0; src < 64; ++src) {
      if (src & 15 & (16 / STEPS - 1)) continue;        // one lane per block of 32 dims
      const int block = (src & 15) / (16 / STEPS);
#pragma nounroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t x = (uint32_t)__builtin_amdgcn_readlane((int)(i < 4 ? t.vs[0] : t.vs[1]), src);
        if (((x >> (8 * (i & 3))) & 255u) != 255u) continue;
        const int tok = base + token(src >> 4, i);
#pragma nounroll
        for (int bit = 0; bit < 4 * M; ++bit) {
          const int mine = (g * (D / 4) + (bit & 3) * (D / 16)) / 32;
          if (mine == block && sees(tok, bit >> 2)) poison |= 1u << bit;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (((t.vs[k >> 2] >> (8 * (k & 3))) & 255u) == 255u) t.vs[k >> 2] ^= 128u << (8 * (k & 3));
  }
  __device__ __forceinline__ void apply_poison() {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (poison >> (16 + mt) & 1) l[mt][0] = __builtin_nanf("");
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (poison >> (4 * mt + r) & 1)
#pragma unroll
          for (int f = 0; f < FR; ++f) o[mt][f][r] = __builtin_nanf("");
    }
  }

  // The wave's tiles: every WAVES-th of the share, for the first M row tiles.
  // id: lane i holds the pages of tile tbegin + i (its two halves).
  static __device__ __forceinline__ int base_of(const Span& sp, int i) {
    return (i < sp.sink_tiles ? i : i - sp.sink_tiles + sp.tile0) * TILE;
  }
  // Lane i: the pages of tile first + i (its two halves), 64 tiles of the share at a time.
  struct Pages {
    int id[2], first;
    // (true if a page is missing or outside the pool; page 0 is read in its place)
    __device__ __forceinline__ bool ask(const AttnArgs& a, const Share& w, const int32_t* tab, int from) {
      const int lane = threadIdx.x & 63;
      bool bad = false;
      first = from;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int slot = (base_of(w.sp, from + lane) + 16 * hf) >> a.page_log2;
        const bool need = from + lane < w.tend && page_needed(w.sp, slot, a.page_log2, a.sinks);
        const bool have = need && slot < a.ld_table;
        id[hf] = tab[have ? slot : 0];
        const bool in_pool = have && (uint32_t)id[hf] < (uint64_t)a.num_pages;
        bad |= need && !in_pool;
        if (!in_pool) id[hf] = 0;
      }
      return __any(bad);
    }
  };
  static __device__ __forceinline__ void fetch(const AttnArgs& a, const Share& w, Tile<D>& t,
                                               const Pages& id, const Lane& at, int i) {
    const uint32_t i0 = (uint32_t)__builtin_amdgcn_readlane(id.id[0], i - id.first);
    const uint32_t i1 = (uint32_t)__builtin_amdgcn_readlane(id.id[1], i - id.first);
    const int tb = base_of(w.sp, i) & (a.page - 1);
    load(t, 0, w.pool + (uint64_t)i0 * w.page_bytes, a.unit, at, tb);
    load(t, 1, w.pool + (uint64_t)i1 * w.page_bytes, a.unit, at, (tb + 16) & (a.page - 1));
  }

  template <int M, int WAVES, bool LONG, int DEPTH>
  __device__ __forceinline__ void run(const AttnArgs& a, const Share& w, Tile<D> (&t)[DEPTH],
                                      Pages& id, const int32_t* tab, bool& bad, const Lane& at, int wave,
                                      const bf16x8* q) {
    const int last = w.tend - 1;
    for (int i = w.tbegin + wave; i < w.tend; i += DEPTH * WAVES) {
#pragma unroll
      for (int k = 0; k < DEPTH; ++k) {
        if (i + k * WAVES < w.tend) {
          const int base = base_of(w.sp, i + k * WAVES);
          const bool masked =
              base + TILE - 1 > w.ctx ||
              (a.window > 0 && base <= w.ctx + w.rows - 1 - a.window && base + TILE > a.sinks);
          step<M>(a, t[k], masked, base, w, q);
        }
        const int ahead = min(i + (k + DEPTH) * WAVES, last);
        if constexpr (LONG)                   // (chunks of more than 64 tiles)
          if (ahead - id.first >= 64) bad |= id.ask(a, w, tab, ahead);
        fetch(a, w, t[k], id, at, ahead);
      }
    }
  }
};

template <typename T, int N>
__device__ __forceinline__ void store_row(T* dst, const float* x) {
  T y[N];
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = (T)x[i];
  __builtin_memcpy(dst, y, sizeof(y));
}

// One workgroup's share: rows from 16 MT rb on, KV head h, one chunk of request b.
struct Item {
  int b, row0, rows, ctx, status, chunk, h, rb;
};

// The items of a call that has room for more than the device runs at once: the
// full chunks of all requests, then the chunks 0, which hold what is left over of
// full ones, by falling work (tiles and row tiles).  So the shortest start last, and
// workgroups without an item come after all others (a batch of ragged contexts has a
// third of the items that its sizes allow).  One workgroup of 1,024, a thread per
// request, then per item.
__global__ __launch_bounds__(1024) void k_attn_plan(AttnArgs a) {
  constexpr int LEVELS = 64;
  __shared__ int wred[2][16], sfull[MAX_BATCH], seach[MAX_BATCH];
  __shared__ int srow0[MAX_BATCH], srows[MAX_BATCH], sctx[MAX_BATCH];
  // chunks 0 by level of work, most first: how many requests (upper half) and items
  __shared__ unsigned long long level[LEVELS + 1];
  __shared__ int order[MAX_BATCH], srest[MAX_BATCH];
  const int b = threadIdx.x, lane = b & 63, wave = b >> 6;
  const int G = a.heads / a.kv_heads;
  int c0 = 0, c1 = 0, ctx = 0, broken = a.batch;
  if (b < a.batch) {
    c0 = a.cu[b];
    c1 = a.cu[b + 1];
    ctx = a.ctx[b];
    if (c0 < 0 || c1 < c0 || c1 > a.total_rows) broken = b;
  }
  if (b < LEVELS) level[b] = 0;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) broken = min(broken, __shfl_xor(broken, d));
  if (lane == 0) wred[0][wave] = broken;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 16; ++w) broken = min(broken, wred[0][w]);
  const int rows = c1 - c0;
  const bool fits = ctx >= 0 && (int64_t)ctx + rows <= a.max_context;
  int full = 0, rest = 0, at_level = LEVELS - 1;
  if (b < broken && rows >= 1 && rows <= a.max_k + 1) {
    rest = a.kv_heads * ((rows * G + a.block_rows - 1) / a.block_rows);
    if (fits) {
      const int tiles = span_of(ctx, rows, a.window, a.sinks).tiles;
      const int ct = chunk_of(a, tiles);
      full = (tiles - 1) / ct * rest;
      // a tile costs about as much as two row tiles' products with it
      const int mt = (min(rows * G, a.block_rows) + 15) / 16, most = a.chunk_tiles * (2 + a.block_rows / 16);
      const int work = min(min((tiles - 1) % ct + 1, a.chunk_tiles) * (2 + mt), most);
      at_level = LEVELS - 1 - work * (LEVELS - 1) / most;
    }
  }
  // (places within a level come as they come: which workgroup computes an item
  // changes nothing in its result)
  const unsigned long long mine = b < a.batch ? atomicAdd(&level[at_level], 1ull << 32 | (unsigned)rest) : 0;
  int f = full;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(f, d);
    if (lane >= d) f += y;
  }
  if (lane == 63) wred[1][wave] = f;
  __syncthreads();
  if (wave == 0) {
    unsigned long long x = level[lane], sum = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const unsigned long long y = __shfl_up(sum, d);
      if (lane >= d) sum += y;
    }
    level[lane] = sum - x;
    if (lane == 63) level[LEVELS] = sum;
  }
  int all_full = 0;
  for (int w = 0; w < 16; ++w) {
    if (w == wave) f += all_full;
    all_full += wred[1][w];
  }
  sfull[b] = f - full;
  seach[b] = rest;
  srow0[b] = c0;
  srows[b] = rows;
  sctx[b] = fits ? ctx : -1;
  __syncthreads();
  const int all = all_full + (int)(unsigned)level[LEVELS];
  if (b < a.batch) {
    const unsigned long long place = level[at_level] + mine;
    order[place >> 32] = b;
    srest[place >> 32] = (int)(unsigned)place;
  }
  if (b == 0) a.plan[0].b = all;
  __syncthreads();
  for (int i = b; i < all; i += 1024) {
    const bool rem = i >= all_full;
    const int* start = rem ? srest : sfull;
    const int at = rem ? i - all_full : i;
    int lo = 0, hi = a.batch;                 // the range that holds it
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= at) lo = mid;
      else hi = mid;
    }
    const int in = at - start[lo];
    if (rem) lo = order[lo];
    const int each = seach[lo], local = in % each, blocks = each / a.kv_heads;
    Item it;
    it.b = lo;
    it.row0 = srow0[lo];
    it.rows = srows[lo];
    it.ctx = max(sctx[lo], 0);
    it.status = sctx[lo] < 0 ? SV_ROW_BAD_PARAM : SV_ROW_OK;
    it.chunk = rem ? 0 : 1 + in / each;
    it.h = local / blocks;
    it.rb = local % blocks;
    a.plan[1 + i] = it;
  }
}

// LONG: with chunks of more than 64 tiles.  (An instance of its own: the check at every
// tile takes 1 % of the verify batch, 2 % of the windowed one.)
template <int D, int MT, int DEPTH, int WAVES, bool LONG, typename T>
__global__ __launch_bounds__(64 * WAVES, 2) void k_attn(AttnArgs a) {
  using A = Attn<D, MT, T>;
  constexpr int FR = A::FR;
  // the query operands, and once all waves are done their results for a row tile
  constexpr int O_BYTES = WAVES * FR * 4 * 64 * 4;
  __shared__ __align__(16) uint8_t smem[O_BYTES > A::Q_BYTES ? O_BYTES : A::Q_BYTES];
  bf16x8* const q_lds = (bf16x8*)smem;
  float (*const part_o)[FR * 4][64] = (float (*)[FR * 4][64])smem;
  __shared__ float part_m[WAVES][MT][16], part_l[WAVES][MT][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int items = a.batch * a.kv_heads * a.row_blocks * a.chunks;
  const int status_blocks = (a.batch + WAVES - 1) / WAVES;

  if ((int)blockIdx.x < status_blocks) {      // a request's status, a wave each
    const int b = (int)blockIdx.x * WAVES + wave;
    if (b >= a.batch) return;
    int row0, rows, ctx;
    int st = request_status(a, b, row0, rows, ctx);
    if (st == SV_ROW_OK) {
      const Span sp = span_of(ctx, rows, a.window, a.sinks);
      const int32_t* tab = a.table + (int64_t)b * a.ld_table;
      bool bad = false;
      for (int s = lane; s <= (sp.n - 1) >> a.page_log2; s += 64)
        if (page_needed(sp, s, a.page_log2, a.sinks))
          bad |= s >= a.ld_table || (uint32_t)tab[s] >= (uint64_t)a.num_pages;
      if (__any(bad)) st = SV_ROW_BAD_PAGE;
    }
    if (lane == 0) a.status[b] = st;
    return;
  }

  int b, row0, rows, ctx, st, chunk, h, rb, it = (int)blockIdx.x - status_blocks;
  if (a.plan) {
    if (it >= a.plan[0].b) return;
    const Item x = a.plan[1 + it];
    b = x.b;
    row0 = x.row0;
    rows = x.rows;
    ctx = x.ctx;
    st = x.status;
    chunk = x.chunk;
    h = x.h;
    rb = x.rb;
  } else {
    rb = it % a.row_blocks;
    it /= a.row_blocks;
    h = it % a.kv_heads;
    it /= a.kv_heads;
    b = it % a.batch;
    chunk = a.chunks - 1 - it / a.batch;
    st = request_status(a, b, row0, rows, ctx);
    if (st == SV_ROW_BAD_K || rb * MT * 16 >= rows * a.group) return;
  }
  Share w;
  w.sp = span_of(ctx, rows, a.window, a.sinks);
  const int ct = LONG ? chunk_of(a, w.sp.tiles) : a.chunk_tiles;
  w.tend = (w.sp.tiles - 1) % ct + 1 + chunk * ct;
  w.tbegin = max(0, w.tend - ct);
  if (st == SV_ROW_OK ? w.tend > w.sp.tiles : chunk > 0) return;
  w.row0 = row0;
  w.ctx = ctx;
  w.rows = rows;
  w.R = rows * a.group;
  w.rb = rb;
  w.c = a.scale * LOG2E;
  w.pool = a.pages + (int64_t)h * a.unit;
  w.page_bytes = (uint32_t)a.unit * (uint32_t)a.kv_heads;
  const int R = w.R;

  A x;
  x.init();
  bool bad = st != SV_ROW_OK;
  if (!bad) {
    const int32_t* tab = a.table + (int64_t)b * a.ld_table;
    typename A::Pages id;
    bad = id.ask(a, w, tab, w.tbegin);
    typename A::template Raw<WAVES> raw;
    raw.ask(a, w, h, wave);
    const typename A::Lane at = A::lane_offsets(a.page);
    // DEPTH tiles are on their way at any time: a buffer is filled again as soon
    // as its tile is done.  Past the end the last tile is loaded once more: with a
    // branch around the loads the compiler could not count those in flight and
    // would wait for all of them at every tile.
    Tile<D> t[DEPTH];
#pragma unroll
    for (int k = 0; k < DEPTH; ++k)
      A::fetch(a, w, t[k], id, at, min(w.tbegin + wave + k * WAVES, w.tend - 1));
    raw.put(q_lds, wave);
    __syncthreads();
    // row tiles that hold rows: a short request does not pay for a long one's
    const int tiles = (min(R - rb * MT * 16, MT * 16) + 15) / 16;
    // (not where the copies of the loop would not fit the registers)
    if (MT * FR >= 32) x.template run<MT, WAVES, LONG>(a, w, t, id, tab, bad, at, wave, q_lds);
    else if (MT == 1 || tiles == 1) x.template run<1, WAVES, LONG>(a, w, t, id, tab, bad, at, wave, q_lds);
    else if (MT == 2 || tiles == 2)
      x.template run<(MT < 2 ? 1 : 2), WAVES, LONG>(a, w, t, id, tab, bad, at, wave, q_lds);
    else if (tiles == 3)
      x.template run<(MT < 3 ? 1 : 3), WAVES, LONG>(a, w, t, id, tab, bad, at, wave, q_lds);
    else x.template run<MT, WAVES, LONG>(a, w, t, id, tab, bad, at, wave, q_lds);
  }
  if (__any(x.poison != 0)) x.apply_poison();

  // join the waves, a row tile at a time: each takes its share of every row's dims
  // (those that are entry r of the accumulators, r = wave + WAVES i)
  const int n = lane & 15, g = lane >> 4;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
    if (g == 0) {
      part_m[wave][mt][n] = x.mc[mt];
      // a page id out of range: the request's rows are NaN
      part_l[wave][mt][n] = bad ? __builtin_nanf("") : x.l[mt][0];
    }

  const bool whole = st != SV_ROW_OK || w.sp.tiles <= ct;
  // this item's place among the partials
  const int64_t item = (((int64_t)chunk * a.batch + b) * a.kv_heads + h) * a.row_blocks + rb;
  float* part = a.part + item * (MT * 16) * D;
  float* stat = a.part + (int64_t)items * (MT * 16) * D + item * (MT * 16) * 2;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    __syncthreads();                          // (every wave is done with what lay here)
#pragma unroll
    for (int f = 0; f < FR; ++f)
#pragma unroll
      for (int r = 0; r < 4; ++r) part_o[wave][f * 4 + r][lane] = x.o[mt][f][r];
    __syncthreads();
    const int r = (rb * MT + mt) * 16 + n;
    float m = part_m[0][mt][n];
#pragma unroll
    for (int k = 1; k < WAVES; ++k) m = fmaxf(m, part_m[k][mt][n]);
    float part_w[WAVES], sum = 0.f;
#pragma unroll
    for (int k = 0; k < WAVES; ++k) {
      const float mk = part_m[k][mt][n];
      part_w[k] = mk == m ? 1.f : __builtin_amdgcn_exp2f(mk - m);
      sum += part_l[k][mt][n] * part_w[k];
    }
    const float inv = 1.f / sum;
    const int j = A::row_of(a, r), hq = h * a.group + r - j * a.group;
#pragma unroll
    for (int q = 0; q < (WAVES < 4 ? 4 / WAVES : 1); ++q) {
      const int e = wave + q * WAVES, dim = g * (D / 4) + e * FR;
      if (e >= 4) continue;                    // (eight waves: four of them join)
      float y[FR];
#pragma unroll
      for (int f = 0; f < FR; ++f) {
        y[f] = 0.f;
#pragma unroll
        for (int k = 0; k < WAVES; ++k)
          y[f] = __builtin_fmaf(part_o[k][f * 4 + e][lane], part_w[k], y[f]);
      }
      if (r >= R) continue;
      if (whole) {
#pragma unroll
        for (int f = 0; f < FR; ++f) y[f] *= inv;
        store_row<T, FR>((T*)a.out + (int64_t)(row0 + j) * a.ld_out + (int64_t)hq * D + dim, y);
      } else {
        store_row<float, FR>(part + (mt * 16 + n) * D + dim, y);
        if (e == 0 && g == 0) {
          stat[(mt * 16 + n) * 2] = m;
          stat[(mt * 16 + n) * 2 + 1] = sum;
        }
      }
    }
  }
}

// Joins the chunks of requests longer than one: a workgroup per row.
template <int D, int MT, typename T>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int E = D / 64, WAVES = 4;       // dims per lane
  __shared__ float red[WAVES][D + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int it = blockIdx.x;
  const int local = it % (MT * 16);          // the row in its item
  it /= MT * 16;
  const int first = it;                      // its item of chunk 0
  const int rb = it % a.row_blocks;
  it /= a.row_blocks;
  const int h = it % a.kv_heads, b = it / a.kv_heads;
  int row0, rows, ctx;
  if (request_status(a, b, row0, rows, ctx) != SV_ROW_OK) return;
  const Span sp = span_of(ctx, rows, a.window, a.sinks);
  const int ct = chunk_of(a, sp.tiles), n = (sp.tiles + ct - 1) / ct;
  const int r = rb * MT * 16 + local;
  if (n < 2 || r >= rows * a.group) return;
  const int64_t per_chunk = (int64_t)a.batch * a.kv_heads * a.row_blocks;
  const float* part = a.part + ((int64_t)first * (MT * 16) + local) * D + lane * E;
  const float* stat = a.part + per_chunk * a.chunks * (MT * 16) * D + ((int64_t)first * (MT * 16) + local) * 2;
  const int64_t step = per_chunk * (MT * 16);
  float m = -INFINITY;
  for (int k = lane; k < n; k += 64) m = fmaxf(m, stat[k * step * 2]);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  // every wave weighs the chunks the same; it adds up every fourth
  float acc[E] = {}, sum = 0.f;
  for (int k0 = 0; k0 < n; k0 += 64) {
    float w = 0.f;
    if (k0 + lane < n) {
      const float mk = stat[(k0 + lane) * step * 2];
      w = mk == m ? 1.f : __builtin_amdgcn_exp2f(mk - m);
      sum += w * stat[(k0 + lane) * step * 2 + 1];
    }
    const int most = min(64, n - k0);
    for (int k1 = wave; k1 < most; k1 += 8 * WAVES) {
      float y[8][E];
#pragma unroll
      for (int u = 0; u < 8; ++u)             // (past the end: the last chunk once more, weight 0)
        __builtin_memcpy(y[u], part + (k0 + min(k1 + u * WAVES, most - 1)) * step * D, sizeof(y[u]));
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int k = k1 + u * WAVES;
        const float wk = __builtin_bit_cast(
            float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), min(k, most - 1)));
        if (k < most)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = __builtin_fmaf(y[u][e], wk, acc[e]);
      }
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
#pragma unroll
  for (int e = 0; e < E; ++e) red[wave][lane * E + e] = acc[e];
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < WAVES; ++w)
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += red[w][lane * E + e];
  const int j = r / a.group, hq = h * a.group + r - j * a.group;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] /= sum;
  store_row<T, E>((T*)a.out + (int64_t)(row0 + j) * a.ld_out + (int64_t)hq * D + lane * E, acc);
}

// The same where rows are many and chunks few: 16 threads per row, 16 rows per
// workgroup, every chunk's part on its way at once.
template <int D, int MT, typename T>
__global__ __launch_bounds__(256) void k_attn_join_rows(AttnArgs a) {
  constexpr int E = D / 16;                  // dims per thread
  const int lane = threadIdx.x & 63, j16 = threadIdx.x & 15;
  const int mt = blockIdx.x % MT, first = blockIdx.x / MT;
  const int rb = first % a.row_blocks, h = first / a.row_blocks % a.kv_heads;
  const int b = first / a.row_blocks / a.kv_heads;
  int row0, rows, ctx;
  if (request_status(a, b, row0, rows, ctx) != SV_ROW_OK) return;
  const Span sp = span_of(ctx, rows, a.window, a.sinks);
  const int ct = chunk_of(a, sp.tiles), n = (sp.tiles + ct - 1) / ct;
  const int local = mt * 16 + (threadIdx.x >> 4), r = rb * MT * 16 + local;
  if (n < 2 || r >= rows * a.group) return;  // (whole groups of 16 lanes)
  const int64_t per_chunk = (int64_t)a.batch * a.kv_heads * a.row_blocks;
  const int64_t step = per_chunk * (MT * 16);
  const float* part = a.part + ((int64_t)first * (MT * 16) + local) * D + j16 * E;
  const float* stat = a.part + step * a.chunks * D + ((int64_t)first * (MT * 16) + local) * 2;
  float m = -INFINITY;
  for (int k = j16; k < n; k += 16) m = fmaxf(m, stat[k * step * 2]);
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  float acc[E] = {}, sum = 0.f;
  for (int k0 = 0; k0 < n; k0 += 16) {
    float w = 0.f;
    if (k0 + j16 < n) {
      const float mk = stat[(k0 + j16) * step * 2];
      w = mk == m ? 1.f : __builtin_amdgcn_exp2f(mk - m);
      sum += w * stat[(k0 + j16) * step * 2 + 1];
    }
    const int most = min(16, n - k0);
    for (int k1 = 0; k1 < most; k1 += 4) {
      float y[4][E];
#pragma unroll
      for (int u = 0; u < 4; ++u)             // (past the end: the last chunk once more, unused)
        __builtin_memcpy(y[u], part + (k0 + min(k1 + u, most - 1)) * step * D, sizeof(y[u]));
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float wk = __shfl(w, (lane & 48) | min(k1 + u, 15));
        if (k1 + u < most)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = __builtin_fmaf(y[u][e], wk, acc[e]);
      }
    }
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor(sum, d);
  const int j = r / a.group, hq = h * a.group + r - j * a.group;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] /= sum;
  store_row<T, E>((T*)a.out + (int64_t)(row0 + j) * a.ld_out + (int64_t)hq * D + j16 * E, acc);
}

// ---- host side

struct Plan {
  int mt, row_blocks, chunks, chunk_tiles, waves;
  size_t part_bytes, bytes;
  bool plan, longer;    // longer: a request can have more tiles than full chunks hold
};

// Of planned calls: two waves per workgroup (more items at once, each twice as long)
// where items are many, and whole or rich in products: 512 requests over 1 to 2,000
// positions 64 us, with four 81; 256 over 1 to 4,000 (R=28) 67.5 and 76.5; 128 over 1 to
// 8,000 with R=56 81.5 and 92; but 64 over 8,000 with R=4 128 and 122, 64 over 1 to 8,000
// at D=256 (one tile on its way per wave) 80 and 61.  fp32 waves take longer for an item
// and need more of them: 512 over 1 to 2,000 79.5 and 97, 256 with R=48 69 and 58.
static constexpr bool two_waves(int dtype, int mt, int d, bool whole, int64_t items) {
  return dtype == SV_F32 ? whole && items >= 4096 : whole || (mt > 1 && d < 256);
}

// What the partial results of a call may take: its bound on contexts is often far above
// what the requests hold, and every place is a workgroup to start.  (256 requests over 200
// to 2,000 positions, k=6, 32 heads over 8 KV heads of D=128, bound 131,072: 488 MiB and
// 93 us, with a place for every chunk 2,084 MiB and 113; 1,024 requests 347 and 441.  One
// request of 131,072 among the 256, in 15 chunks of 274 tiles: 164 us, in 64 157.)
constexpr int64_t PLACES = 512ll << 20;

// Rows per workgroup and the split over the context, by the call's sizes alone.
static bool plan_of(int dtype, int batch, int max_k, int heads, int kv_heads, int d,
                    int max_context, int window, int sinks, Plan& p) {
  const int64_t R = (int64_t)(max_k + 1) * (heads / kv_heads);
  // tiles a request can have: two borders more than its tokens fill
  int64_t tokens = max_context;
  if (window > 0) {
    const int64_t seen = (int64_t)window + max_k + 1 + sinks + 3 * TILE;
    if (seen < tokens) tokens = seen;
  }
  const int64_t tiles = (tokens + TILE - 1) / TILE;
  // what fits the vector registers; tests/test_kernel_registers.py holds every instance
  // to it.  The compiler (clang 22.0.0git, roc-7.2.0) made a wrong kernel of one that
  // did not fit: 32 rows at D=256 with two tiles on their way spilled 113 registers, the
  // four words of row tile 1's first query operand among them, two to scratch and two to
  // accumulation registers, of which only one was read back before the matrix
  // instructions, so that rows 16 to 31 were wrong.  (64 requests over 2,000 positions, R=28, D=256: 65
  // us with 32 rows per workgroup, 93 with 16.  64 rows at D=128, K widened for each
  // row tile again to fit: R=56, 64 over 4,000 116 us, with 32 rows 130; but 128 over 1
  // to 8,000 99 and 82, 8 over 4,000 30 and 27.)
  const int most = dtype == SV_BF16 && d == 256 ? 2 : 256 / d;
  p.mt = R <= 16 ? 1 : R <= 32 ? 2 : 4;
  if (p.mt > most) p.mt = most;
  int64_t items;
  for (;; p.mt = 1) {
    p.row_blocks = (int)((R + p.mt * 16 - 1) / (p.mt * 16));
    const int64_t wide = (int64_t)batch * kv_heads * p.row_blocks;
    // chunks of 64 tiles (a lane of a wave each), halved down to 256 tokens while
    // there is less than a workgroup per compute unit.  (One user over 32,000
    // positions: 18.5 us with 256 workgroups, 21.5 with 512, 26 with 1,024.)
    int64_t ct = 64;
    while (ct > 8 && wide * ((tiles + ct - 1) / ct) < 256) ct /= 2;
    p.chunk_tiles = (int)ct;
    // a place for the partial results of every chunk that the sizes allow, up to 512 MiB
    // or 8 chunks per request: those who would have more get longer ones
    const int64_t places = PLACES / (wide * p.mt * 16 * (d + 2) * (int64_t)sizeof(float));
    const int64_t chunks = (tiles + ct - 1) / ct, room = places < 8 ? 8 : places;
    p.chunks = (int)(chunks < room ? chunks : room);
    p.longer = chunks > room;
    items = wide * p.chunks;
    // fp32 rows cost a wave three times the products: where workgroups are few, its
    // time is that of the longest wave, and 16 rows each are better (R=24: 32 requests
    // over 1 to 2,000 positions 16.0 us, with 32 rows 22; 64 over 2,000 73 and 60)
    if (p.mt == 1 || dtype != SV_F32 || items >= 512) break;
  }
  // (a launch has less than 2^32 threads)
  if (items >= (1ll << 24) - MAX_BATCH) return false;
  p.part_bytes = p.chunks > 1 ? (size_t)items * (p.mt * 16) * (d + 2) * sizeof(float) : 0;
  p.plan = items > 1024;
  p.waves = p.plan && two_waves(dtype, p.mt, d, p.chunks == 1, items) ? 2 : 4;
  // eight for fp32, whose waves are the slowest, where workgroups are few (32 requests
  // over 1 to 2,000 positions 16.1 us, with four 18.0; 8 over 2,000 19.5 both ways).
  // bf16 only loses by the longer join (4 over 500: 13.4 us against 12.0), and at
  // D=256 the waves have no registers left to overlap (29.0 us against 28.1)
  if (items < 512 && dtype == SV_F32 && d < 256) p.waves = 8;    // (p.mt is 1)
  p.bytes = p.part_bytes + (p.plan ? (size_t)(items + 1) * sizeof(Item) : 0);
  return true;
}

static bool sizes_ok(int dtype, int batch, int max_k, int heads, int kv_heads, int d,
                     int max_context, int window, int sinks) {
  return (dtype == SV_F32 || dtype == SV_BF16) && batch >= 1 && batch <= MAX_BATCH && max_k >= 0 &&
         max_k <= 63 && kv_heads >= 1 && heads >= kv_heads && heads % kv_heads == 0 &&
         heads <= 1024 && dim_ok(d) && max_context >= 1 && max_context <= (1 << 30) &&
         window >= 0 && window <= (1 << 30) && sinks >= 0 && sinks <= (1 << 30);
}

template <int D, int MT, int DEPTH, typename T>
static int launch(const AttnArgs& a, const Plan& p, hipStream_t s) {
  const int items = a.batch * a.kv_heads * p.row_blocks * p.chunks;
  if (a.plan) {
    hipLaunchKernelGGL(k_attn_plan, dim3(1), dim3(1024), 0, s, a);
    if (hipGetLastError() != hipSuccess) return SV_ERR_LAUNCH;
  }
  const int grid = items + (a.batch + p.waves - 1) / p.waves;
  if (p.longer) {                             // (planned, with several chunks: see plan_of)
    constexpr int WAVES = two_waves(sizeof(T) == 4 ? SV_F32 : SV_BF16, MT, D, false, 0) ? 2 : 4;
    hipLaunchKernelGGL((k_attn<D, MT, DEPTH, WAVES, true, T>), dim3(grid), dim3(64 * WAVES), 0, s, a);
  } else if (p.waves == 2) {
    hipLaunchKernelGGL((k_attn<D, MT, DEPTH, 2, false, T>), dim3(grid), dim3(128), 0, s, a);
  } else if (p.waves == 4) {
    hipLaunchKernelGGL((k_attn<D, MT, DEPTH, 4, false, T>), dim3(grid), dim3(256), 0, s, a);
  } else {
    if constexpr (sizeof(T) == 4 && D < 256 && MT == 1)
      hipLaunchKernelGGL((k_attn<D, MT, DEPTH, 8, false, T>), dim3(grid), dim3(512), 0, s, a);
  }
  if (hipGetLastError() != hipSuccess) return SV_ERR_LAUNCH;
  if (p.chunks > 1) {
    const int wide = a.batch * a.kv_heads * p.row_blocks;
    // a workgroup per row where few rows have many chunks (one user over 32,000
    // positions: 18.5 us a call, with the other form 22), else per 16 rows (8
    // requests over 2,000: 16.5 us, a workgroup per row 20.8)
    if (p.chunks > 8 && wide * MT * 16 <= 2048)
      hipLaunchKernelGGL((k_attn_join<D, MT, T>), dim3(wide * (MT * 16)), dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((k_attn_join_rows<D, MT, T>), dim3(wide * MT), dim3(256), 0, s, a);
    if (hipGetLastError() != hipSuccess) return SV_ERR_LAUNCH;
  }
  return SV_OK;
}

}  // namespace svk

using namespace svk;

extern "C" {

size_t spec_kv_attention_workspace_bytes(int dtype, int batch, int max_k, int heads, int kv_heads,
                                         int head_dim, int max_context, int window, int sinks) {
  Plan p;
  if (!sizes_ok(dtype, batch, max_k, heads, kv_heads, head_dim, max_context, window, sinks) ||
      !plan_of(dtype, batch, max_k, heads, kv_heads, head_dim, max_context, window, sinks, p))
    return 0;
  return p.bytes > 16 ? p.bytes : 16;
}

int spec_kv_attention(const void* q, int64_t ld_q, int dtype, const int32_t* cu_seqlens,
                      const int32_t* context_lens, int batch, int total_rows, int max_k, int heads,
                      int kv_heads, int head_dim, const void* pages, int64_t num_pages,
                      int page_size, const int32_t* page_table, int64_t ld_table, int max_context,
                      float scale, int window, int sinks, void* out, int64_t ld_out,
                      int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !cu_seqlens || !context_lens || !pages || !page_table || !out || !status)
    return SV_ERR_NULL;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  Plan p;
  if (!sizes_ok(dtype, batch, max_k, heads, kv_heads, head_dim, max_context, window, sinks) ||
      total_rows < 1 || !page_ok(page_size) || num_pages < 1 || num_pages > 0x7fffffff ||
      ld_table < 1 || ld_table > (1 << 30) / page_size || ld_q < (int64_t)heads * head_dim ||
      ld_out < (int64_t)heads * head_dim || !(scale > 0.f) || !(scale <= 2.0e38f) ||
      !aligned16(pages) ||
      !plan_of(dtype, batch, max_k, heads, kv_heads, head_dim, max_context, window, sinks, p))
    return SV_ERR_SHAPE;
  if (p.bytes && (!workspace || !aligned16(workspace))) return SV_ERR_NULL;
  if (p.bytes > workspace_bytes) return SV_ERR_WORKSPACE;
  AttnArgs a;
  a.q = q;
  a.ld_q = ld_q;
  a.cu = cu_seqlens;
  a.ctx = context_lens;
  a.batch = batch;
  a.total_rows = total_rows;
  a.max_k = max_k;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.group = heads / kv_heads;
  a.inv_group = 1.f / (float)a.group;
  a.unit = (int)unit_bytes(page_size, head_dim);
  a.pages = (const uint8_t*)pages;
  a.num_pages = num_pages;
  a.page = page_size;
  a.page_log2 = __builtin_ctz((unsigned)page_size);
  a.table = page_table;
  a.ld_table = ld_table;
  a.max_context = max_context;
  a.scale = scale;
  a.window = window;
  a.sinks = sinks;
  a.out = out;
  a.ld_out = ld_out;
  a.status = status;
  a.part = (float*)workspace;
  a.chunks = p.chunks;
  a.chunk_tiles = p.chunk_tiles;
  a.row_blocks = p.row_blocks;
  a.block_rows = p.mt * 16;
  a.plan = p.plan ? (Item*)((uint8_t*)workspace + p.part_bytes) : nullptr;
  hipStream_t s = (hipStream_t)stream;
#define SVK_CASE(DD, MM, KK, TT) \
  if (head_dim == DD && p.mt == MM) return launch<DD, MM, KK, TT>(a, p, s)
  if (dtype == SV_BF16) {
    SVK_CASE(64, 1, 3, __bf16);
    SVK_CASE(64, 2, 2, __bf16);
    SVK_CASE(64, 4, 2, __bf16);
    SVK_CASE(128, 1, 3, __bf16);
    SVK_CASE(128, 2, 2, __bf16);
    SVK_CASE(256, 2, 1, __bf16);
    SVK_CASE(256, 1, 2, __bf16);
  } else {
    SVK_CASE(64, 1, 2, float);
    SVK_CASE(128, 1, 2, float);
    SVK_CASE(256, 1, 2, float);
    SVK_CASE(128, 2, 2, float);
    SVK_CASE(64, 2, 2, float);
    SVK_CASE(64, 4, 1, float);
  }
#undef SVK_CASE
  return SV_ERR_SHAPE;
}

}  // extern "C"
