// One warp's attention state over an 8-bit cache: up to NT * 8 query rows of
// one KV head, blocks of 16 tokens from shared-memory tiles.
//
// Mathematics.  With byte values k8, v8 and a block's scales ks, vs:
//   x = (q . k8) * (scale * log2 e * ks)              scores in log2 units
//   M = running max of x + log2 vs,  p = 2^(x - M + 15)
//   l += p,   O += (p vs) v8,   out = O / l.
// Putting log2 vs into the reference keeps every weight p vs at or below
// 2^15 whatever the scales of different blocks are, so the weights fit f16
// (normal down to 2^-29 of the largest) and a block's scale never touches O.
//
// Tensor cores: m16n8k16 with f16 operands and fp32 sums.  e4m3 values are
// exact in f16, and so is a bf16 query row once it is multiplied by the power
// of two that brings its largest element to 2^14 .. 2^15 (undone in the score's
// factor).  Weights are rounded to f16 (11 bits, where a bf16 output has 8).
// fp32 queries and weights are split in two f16 terms (22 bits): HILO.
//
// Tokens and head dims are the 16 rows of the A operand and the query rows
// the 8 columns of B, so eight query heads of a KV head fill a tile.
//   S^T [16 tokens x 8 rows] = K Q^T.  The order of the head dims within the
//     product is free: lane (g, c) holds 16 consecutive bytes of tokens g and
//     g + 8, one vector load each, and Q is permuted alike.
//   P^T goes from the accumulator to the B operand by a transposing
//     movmatrix.
//   O^T [16 dims x 8 rows] += V^T P^T.  Lane (g, c) holds HD / 8 consecutive
//     dims of tokens 2c, 2c + 1, 2c + 8, 2c + 9; byte permutes pair the tokens.
// The token order within a block is free too (kTok): it is chosen so that
// both loads touch each bank once in the tile's swizzled layout (heads of 64
// and 128; narrower ones at worst twice).
#pragma once

#include <climits>

#include "device.cuh"
#include "fp8.cuh"

namespace pkv {
namespace fp8 {

constexpr int kBS = 16;
constexpr float kWeightLog2 = 15.f;  // log2 of the largest weight
constexpr float kSumStep = 100.f;    // the sum is scaled by at most 2^-100 at once

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 unpack_f16x2(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// A block's tile in shared memory: rows of `width` bytes (the TMA box's inner
// extent), 16 rows (tokens) for each run of `width` bytes of the group's heads.
// Rows are as wide as they can be, up to 128 bytes, since TMA moves about one
// row in four cycles whatever its width: at head_dim 64 two heads share one.
// The 16-byte piece i of token t sits at piece i ^ swz(t) (the hardware's
// swizzle of that width).
struct TileView {
  int width;

  static __host__ __device__ int swizzle(int width) { return width >= 64 ? width : 0; }
  __device__ __forceinline__ int swz(int t) const {
    return width == 128 ? (t & 7) : width == 64 ? ((t >> 1) & 3) : 0;
  }
  // Byte, within the tile, of byte b of the group's row of token t.
  __device__ __forceinline__ int at(int t, int b) const {
    const int run = b / width, o = b - run * width;
    return (run * kBS + t) * width + (((o >> 4) ^ swz(t)) << 4) + (o & 15);
  }
  // Token of MMA row i (rows i + 8: token + 8), eight 4-bit entries.
  __device__ __forceinline__ int tok(int i) const {
    const uint32_t order = width == 128  ? 0x37156240u   // 0 4 2 6 5 1 7 3
                           : width == 64 ? 0x65742130u   // 0 3 1 2 4 7 5 6
                           : width == 32 ? 0x57463120u   // 0 2 1 3 6 4 7 5
                                         : 0x76543210u;
    return static_cast<int>((order >> (4 * i)) & 15u);
  }
};

// Widest row that whole rows of `heads` heads divide into.
inline int tile_width(int heads, int head_dim) {
  int w = 128;
  while ((heads * head_dim) % w != 0) w /= 2;
  return w;
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&x)[4]);
template <>
__device__ __forceinline__ void load4<float>(const float* p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
}

// CAUSAL: rows may see different last keys (a prefill chunk).
template <typename T, int HD, int NT, bool CAUSAL>
struct Rows {
  static constexpr bool HILO = sizeof(T) == 4;
  static constexpr int PARTS = HILO ? 2 : 1;
  static constexpr int KK = HD / 16;                  // k steps of Q K^T, m tiles of V^T P^T
  static constexpr int KB = HD / 4 < 16 ? HD / 4 : 16;  // bytes of a K piece a lane loads
  static constexpr int NK = HD / 4 / KB;              // K pieces of a token per lane
  static constexpr int DB = HD / 8;                   // dims of V^T a lane holds
  static constexpr int VW = DB / 4 > 0 ? DB / 4 : 1;  // 32-bit words of them
  // blocks taken together, as the registers allow
  static constexpr int PAIR = HD * NT * PARTS <= 128 ? 2 : 1;

  uint32_t qb[NT][PARTS][KK][2];
  float o[NT][KK][4];
  float m[NT][2], l[NT][2], rs[NT][2];
  int last[NT][2];
  int cut;  // least last key over the active rows
  TileView tile;
  int head_off;             // the head's first byte in the group's row
  int koff[NK], voff[2];    // this lane's pieces of K and V in a tile
  int tok_k, tok_v[2];      // their tokens

  // Where the warp's head lies in the tiles.
  __device__ __forceinline__ void place(int width, int head) {
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    tile.width = width;
    head_off = head * HD;
    tok_k = tile.tok(g);
#pragma unroll
    for (int i = 0; i < NK; ++i) koff[i] = tile.at(tok_k, head_off + i * 64 + c * KB);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      tok_v[i] = tile.tok(2 * c + i);
      voff[i] = tile.at(tok_v[i], head_off + g * DB);
    }
  }

  // q_row(r): row r's query (null: no such row); last_key(r): the last key
  // it sees (-1: none).
  template <typename QRow, typename LastKey>
  __device__ __forceinline__ void begin(QRow q_row, LastKey last_key, float scale_log2) {
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    int least = INT_MAX;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[KK][4];
      const T* qp = q_row(nt * 8 + g);
      float a = 0.f;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        // the dims of the K word that step kk multiplies
        const int d = (kk / (KB / 4)) * 64 + c * KB + (kk % (KB / 4)) * 4;
        x[kk][0] = x[kk][1] = x[kk][2] = x[kk][3] = 0.f;
        if (qp) load4<T>(qp + d, x[kk]);
#pragma unroll
        for (int e = 0; e < 4; ++e) a = fmaxf(a, fabsf(x[kk][e]));
      }
      a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
      a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
      // the power of two that brings the row's largest element to 2^14 .. 2^15
      const int up = min(126, 14 + 127 - static_cast<int>(__float_as_uint(a) >> 23));
      const float f = pow2f(up);
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x0 = x[kk][2 * e] * f, x1 = x[kk][2 * e + 1] * f;
          qb[nt][0][kk][e] = pack_f16x2(x0, x1);
          if constexpr (HILO) {
            const float2 hi = unpack_f16x2(qb[nt][0][kk][e]);
            qb[nt][1][kk][e] = pack_f16x2(x0 - hi.x, x1 - hi.y);
          }
        }
      const float back = pow2f(-up) * scale_log2;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = nt * 8 + 2 * c + j;
        rs[nt][j] = __shfl_sync(0xffffffffu, back, (2 * c + j) * 4);
        // a row without a query is never masked (and never stored)
        last[nt][j] = q_row(r) ? last_key(r) : INT_MAX;
        least = min(least, last[nt][j]);
        m[nt][j] = -INFINITY;
        l[nt][j] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < KK; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }
    cut = __reduce_min_sync(0xffffffffu, least);
  }

  // NB consecutive blocks: their K and V tiles, the position j0 of the first
  // token, the sequence's tokens from there on (valid: V rows past them are not
  // used), the blocks' scales and lv = log2 vs.  Two at a time share one
  // maximum, one rescaling and the latency of each step.
  template <int NB>
  __device__ __forceinline__ void blocks(const uint8_t* const (&kt)[NB],
                                         const uint8_t* const (&vt)[NB], int j0, int valid,
                                         const float (&ks)[NB], const float (&vs)[NB],
                                         const float (&lv)[NB]) {
    // ---- S^T = K Q^T, two chains of products
    uint32_t vw[NB][4][VW];  // tokens tok(2c), tok(2c + 1), and those + 8
    float w[NB][NT][4];      // scores, then weights
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      uint32_t kw[2][KK];  // [token g | g + 8]: words of 4 dims
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < NK; ++i) {
          const uint8_t* p = kt[nb] + koff[i] + h * 8 * tile.width;
          if constexpr (KB == 16) {
            const uint4 x = *reinterpret_cast<const uint4*>(p);
            kw[h][4 * i] = x.x, kw[h][4 * i + 1] = x.y, kw[h][4 * i + 2] = x.z, kw[h][4 * i + 3] = x.w;
          } else if constexpr (KB == 8) {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            kw[h][0] = x.x, kw[h][1] = x.y;
          } else {
            kw[h][0] = *reinterpret_cast<const uint32_t*>(p);
          }
        }
      // V's words too: in flight while the scores are computed
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const uint8_t* p = vt[nb] + voff[h & 1] + (h >> 1) * 8 * tile.width;
        if constexpr (DB == 16) {
          const uint4 x = *reinterpret_cast<const uint4*>(p);
          vw[nb][h][0] = x.x, vw[nb][h][1] = x.y, vw[nb][h][2] = x.z, vw[nb][h][3] = x.w;
        } else if constexpr (DB == 8) {
          const uint2 x = *reinterpret_cast<const uint2*>(p);
          vw[nb][h][0] = x.x, vw[nb][h][1] = x.y;
        } else if constexpr (DB == 4) {
          vw[nb][h][0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
          vw[nb][h][0] = *reinterpret_cast<const uint16_t*>(p);
        }
      }
      constexpr int CH = KK >= 4 ? 2 : 1;
      float s[NT][CH][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < CH; ++i) s[nt][i][0] = s[nt][i][1] = s[nt][i][2] = s[nt][i][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        const uint32_t a0 = e4m3x2_to_f16x2(static_cast<uint16_t>(kw[0][kk]));
        const uint32_t a1 = e4m3x2_to_f16x2(static_cast<uint16_t>(kw[1][kk]));
        const uint32_t a2 = e4m3x2_to_f16x2(static_cast<uint16_t>(kw[0][kk] >> 16));
        const uint32_t a3 = e4m3x2_to_f16x2(static_cast<uint16_t>(kw[1][kk] >> 16));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int pt = 0; pt < PARTS; ++pt)
            mma_f16_16816(s[nt][kk % CH], a0, a1, a2, a3, qb[nt][pt][kk][0], qb[nt][pt][kk][1]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = s[nt][0][e];
          if constexpr (CH == 2) x += s[nt][1][e];
          w[nb][nt][e] = x * (rs[nt][e & 1] * ks[nb]);
        }
    }
    // ---- mask, running maximum, weights
    const bool masked = j0 + NB * kBS - 1 > cut;
    if (masked) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j0 + nb * kBS + tok_k + (e >> 1) * 8 > last[nt][e & 1]) w[nb][nt][e] = -INFINITY;
    }
    // d: log2 of the factor on what came before; f: that of the sum
    float d[NT][2], f[NT][2], sum[NT][2];
    bool moved = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float mx = fmaxf(w[0][nt][j], w[0][nt][2 + j]) + lv[0];
#pragma unroll
        for (int nb = 1; nb < NB; ++nb) mx = fmaxf(mx, fmaxf(w[nb][nt][j], w[nb][nt][2 + j]) + lv[nb]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float mn = fmaxf(m[nt][j], mx);
        const float ref = mn == -INFINITY ? 0.f : mn;  // nothing visible yet
        d[nt][j] = m[nt][j] - ref;
        moved |= mn != m[nt][j];
        m[nt][j] = mn;
        f[nt][j] = 1.f;
        sum[nt][j] = 0.f;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float p0 = fast_exp2(w[nb][nt][j] - (ref - kWeightLog2));
          const float p1 = fast_exp2(w[nb][nt][2 + j] - (ref - kWeightLog2));
          sum[nt][j] += p0 + p1;
          w[nb][nt][j] = p0 * vs[nb];
          w[nb][nt][2 + j] = p1 * vs[nb];
        }
      }
    // The outputs are rescaled only when some row's maximum moved.  The sum's
    // factor is applied in two steps: 2^d underflows where a block's value scale
    // is some 2^100 times the earlier ones', whose keys then still count in l
    // (their weights p are as large as their scales are small).
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float a0 = fast_exp2(d[nt][0]), a1 = fast_exp2(d[nt][1]);
#pragma unroll
        for (int i = 0; i < KK; ++i) {
          o[nt][i][0] *= a0;
          o[nt][i][1] *= a1;
          o[nt][i][2] *= a0;
          o[nt][i][3] *= a1;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          l[nt][j] *= fast_exp2(fminf(d[nt][j] + kSumStep, 0.f));
          f[nt][j] = fast_exp2(fmaxf(d[nt][j], -kSumStep));
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) l[nt][j] = l[nt][j] * f[nt][j] + sum[nt][j];
    // V rows past the sequence's end hold whatever the pool holds there
    if (valid < NB * kBS) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (nb * kBS + tok_v[h & 1] + (h >> 1) * 8 >= valid)
#pragma unroll
            for (int i = 0; i < VW; ++i) vw[nb][h][i] = 0u;
    }
    bool by_term = false;
    if constexpr (CAUSAL) {
      // a NaN among the values must not reach the rows that do not see its
      // token, as it would through 0 * NaN in the product: such blocks are
      // summed term by term
      bool nan = false;
      if (masked) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int i = 0; i < VW; ++i)
              nan |= __vcmpeq4(vw[nb][h][i] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
      }
      by_term = __any_sync(0xffffffffu, nan);
    }
    // ---- O^T += V^T P^T
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if (CAUSAL && by_term) {
        add_by_term(vt[nb], w[nb], j0 + nb * kBS, valid - nb * kBS);
        continue;
      }
      uint32_t pb[NT][PARTS][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t hi = pack_f16x2(w[nb][nt][2 * h], w[nb][nt][2 * h + 1]);
          pb[nt][0][h] = transpose_8x8(hi);
          if constexpr (HILO) {
            const float2 f = unpack_f16x2(hi);
            pb[nt][1][h] =
                transpose_8x8(pack_f16x2(w[nb][nt][2 * h] - f.x, w[nb][nt][2 * h + 1] - f.y));
          }
        }
#pragma unroll
      for (int i = 0; i < VW; ++i)
#pragma unroll
        for (int half = 0; half < (DB >= 4 ? 2 : 1); ++half) {
          const uint32_t sel = half == 0 ? 0x5140u : 0x7362u;
          const uint32_t lo = __byte_perm(vw[nb][0][i], vw[nb][1][i], sel);
          const uint32_t hi = __byte_perm(vw[nb][2][i], vw[nb][3][i], sel);
          const uint32_t a0 = e4m3x2_to_f16x2(static_cast<uint16_t>(lo));
          const uint32_t a1 = e4m3x2_to_f16x2(static_cast<uint16_t>(lo >> 16));
          const uint32_t a2 = e4m3x2_to_f16x2(static_cast<uint16_t>(hi));
          const uint32_t a3 = e4m3x2_to_f16x2(static_cast<uint16_t>(hi >> 16));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int pt = 0; pt < PARTS; ++pt)
              mma_f16_16816(o[nt][2 * i + half], a0, a1, a2, a3, pb[nt][pt][0], pb[nt][pt][1]);
        }
    }
  }

  // O += P V of a masked block term by term, the terms of hidden tokens left
  // out (w is 0 there but the value may be NaN).
  __device__ __forceinline__ void add_by_term(const uint8_t* vt, const float (&w)[NT][4], int j0,
                                           int valid) {
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
#pragma unroll 1
    for (int ti = 0; ti < kBS; ++ti) {
      const int t = tile.tok(ti & 7) + (ti & 8);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float wj = __shfl_sync(0xffffffffu, ti < 8 ? w[nt][j] : w[nt][2 + j],
                                       (ti & 7) * 4 + c);
          if (t >= valid || j0 + t > last[nt][j]) continue;
#pragma unroll
          for (int i = 0; i < KK; ++i) {
            const int d = g * DB + 2 * i;
            const uint16_t v2 = *reinterpret_cast<const uint16_t*>(vt + tile.at(t, head_off + d));
            const float2 v = e4m3x2_to_float2(v2);
            o[nt][i][j] = fmaf(wj, v.x, o[nt][i][j]);
            o[nt][i][2 + j] = fmaf(wj, v.y, o[nt][i][2 + j]);
          }
        }
    }
  }

  __device__ __forceinline__ void reduce_sums() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 4);
        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 8);
        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 16);
      }
  }

  // Output of every row: out_row(r) -> T* (null: skip).  A row that sees no
  // key gets zeros.
  template <typename OutRow>
  __device__ __forceinline__ void store(OutRow out_row) {
    reduce_sums();
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        T* op = out_row(nt * 8 + 2 * c + j);
        if (!op) continue;
        op += g * DB;
        const float inv = l[nt][j] == 0.f ? 0.f : 1.f / l[nt][j];
        float x[DB];
#pragma unroll
        for (int i = 0; i < KK; ++i) {
          x[2 * i] = o[nt][i][j] * inv;
          x[2 * i + 1] = o[nt][i][2 + j] * inv;
        }
        if constexpr (HILO) {
          store_f32(op, x);
        } else if constexpr (DB >= 8) {
#pragma unroll
          for (int i = 0; i < DB / 8; ++i)
            reinterpret_cast<uint4*>(op)[i] =
                make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                           pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
        } else if constexpr (DB == 4) {
          *reinterpret_cast<uint2*>(op) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        } else {
          *reinterpret_cast<uint32_t*>(op) = pack_bf16x2(x[0], x[1]);
        }
      }
  }

  static __device__ __forceinline__ void store_f32(float* op, const float (&x)[DB]) {
    if constexpr (DB >= 4) {
#pragma unroll
      for (int i = 0; i < DB / 4; ++i)
        reinterpret_cast<float4*>(op)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
      *reinterpret_cast<float2*>(op) = make_float2(x[0], x[1]);
    }
  }

  // Partial result of every row: normalised output (fp32), the reference of
  // its sum in log2 units and the sum.  A sum far from 1, as value scales far
  // from 1 make it, hands its exponent to the reference: the difference of two
  // parts' references is then that of what they weigh, and does not underflow in
  // a merge for a part that counts.  A NaN sum is passed on as NaN outputs with a
  // sum of 1, so that a merge that drops parts without weight keeps it.
  template <typename PartRow, typename MlRow>
  __device__ __forceinline__ void store_partial(PartRow part_row, MlRow ml_row) {
    reduce_sums();
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = nt * 8 + 2 * c + j;
        float* pp = part_row(r);
        if (!pp) continue;
        const bool bad = !(l[nt][j] >= 0.f);
        const float inv = bad ? NAN : l[nt][j] == 0.f ? 0.f : 1.f / l[nt][j];
        float x[DB];
#pragma unroll
        for (int i = 0; i < KK; ++i) {
          x[2 * i] = o[nt][i][j] * inv;
          x[2 * i + 1] = o[nt][i][2 + j] * inv;
        }
        store_f32(pp + g * DB, x);
        if (g == 0) {
          float* ml = ml_row(r);
          int e = static_cast<int>(__float_as_uint(l[nt][j]) >> 23) - 127;
          if (abs(e) <= 40 || l[nt][j] == 0.f) e = 0;
          ml[0] = bad ? 0.f : m[nt][j] + static_cast<float>(e);
          ml[1] = bad ? 1.f : l[nt][j] * pow2f(-e);
        }
      }
  }
};

}  // namespace fp8
}  // namespace pkv
