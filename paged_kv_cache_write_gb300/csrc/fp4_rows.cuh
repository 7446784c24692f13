// One warp's attention state over a 4-bit cache: up to NT * 8 query rows of one KV
// head, blocks of 16 tokens from shared-memory tiles.
//
// Mathematics.  With k4, v4 the products of code and group scale (exact f16 numbers)
// and kg, vg the head's scales:
//   x = (q . k4) * (scale * log2 e * kg)      scores in log2 units
//   p = 2^(x - M + 4),  l += p,   O += p v4,   out = vg O / l.
// The head's scales are constants of a warp, so they cost nothing per key.  M is a
// running reference, the maximum of x when it was last set: weights are computed
// against it as it stands, and only if they come out past f16's range (the maximum has
// grown 2^12-fold: seldom after the first block) is the maximum taken, the reference
// moved to it and what came before rescaled.  Weights are f16 numbers, normal down to
// 2^-18 of the reference's.
//
// Tensor cores: m16n8k16 with f16 operands and fp32 sums.  A bf16 query row is exact
// in f16 once it is multiplied by the power of two that brings its largest element
// to 2^14 .. 2^15 (undone in the score's factor).  Weights are rounded to f16 (11
// bits, where a bf16 output has 8).  fp32 queries and weights are split in two f16
// terms (22 bits): HILO.  A query's second term ends at f16's 2^-24, which is 2^-38 of its
// row's largest element.  A weight's would end at 2^-28 of the reference's, and lose what
// many small weights have in common (1,024 equal ones 2^-17 of the first: 1e-4), so it is
// taken times 2^11 and its product with V divided by that: 22 bits down to 2^-18 (64
// sequences of 512 - 2,048 tokens, 32 heads on 8 of 64, 29.7 us for 28.2; prefill of 4 chunks
// of 256 at the end of 1,000 tokens, 8 heads on 4 of 128, 88.7 for 83.2).
// The tensor cores cut their sums off instead of rounding them, and over a long sequence
// that adds up, so for fp32 each block's product is added to the output by itself: of 2,048
// tokens of heads of 128, 256 queries each, outputs are off by 0.97e-6 for 4.8e-6, in 164 us
// for 145.  (The scores' products too: 0.51e-6, 181 us.)  A bf16 output loses some 2^-23 for
// every 16 tokens that are added up in a row, 6.5e-4 over 131,072: below its half step,
// 2^-8, up to some 500,000.
//
// Tokens and head dims are the 16 rows of the A operand and the query rows the 8
// columns of B, so eight query heads of a KV head fill a tile.
//   S^T [16 tokens x 8 rows] = K Q^T.  The order of the head dims within the product
//     is free: lane (g, c) holds HD / 4 consecutive dims of tokens g and g + 8, one
//     vector load each, and Q is permuted alike.  A word of eight codes is four
//     conversions and four products with the group's scale.
//   P^T goes from the accumulator to the B operand by a transposing movmatrix.
//   O^T [16 dims x 8 rows] += V^T P^T.  Lane (g, c) holds HD / 8 consecutive dims of
//     tokens 2c, 2c + 1, 2c + 8, 2c + 9.  An operand register is one dim of two tokens:
//     their words are merged nibble by nibble first (two operations for four
//     registers), so that one conversion gives the pair.
// Per block and head of 64 that is some 54 instructions for the scores, 74 for the output
// and 24 for the softmax; a warp's chain through them takes 0.55 us a block, whatever else
// the SM does.
//
// The token order within a block is free too (tok): rows of a head are 64 bytes (HD
// 128) or 32, and it is chosen so that K's loads touch each bank once, V's at 64
// bytes twice (half of the banks lie in each row's other half).
#pragma once

#include <climits>

#include "fp4.cuh"
#include "fp8_rows.cuh"

namespace pkv {
namespace fp4 {

using fp8::kBS;
using fp8::load4;
using fp8::mma_f16_16816;
using fp8::pack_f16x2;
using fp8::transpose_8x8;
using fp8::unpack_f16x2;

constexpr float kWeightLog2 = 4.f;     // log2 of the reference's weight
constexpr float kWeightMax = 65504.f;  // f16's largest
// An fp32 weight's second term times 2^11: at most 2^4, half a step of the largest f16
// number, so it stays within f16, and is a normal number where the first term is one.
constexpr float kLowUp = 2048.f, kLowDown = 1.f / 2048.f;
// No reference yet: below every score that fp32 holds by more than it rounds away, so
// that a visible key's weight comes out infinite and a hidden one's (-inf) zero.
constexpr float kNone = -3.0e38f;

// A head's block in shared memory: K codes, V codes, K scales, V scales as they lie in
// the pools, each [16 tokens][..].
template <int HD>
struct Tile {
  static constexpr int kCodes = kBS * HD / 2, kGroups = kBS * HD / kGroup;
  static constexpr int kVCodes = kCodes, kKGroups = 2 * kCodes, kVGroups = 2 * kCodes + kGroups;
  static constexpr int kBytes = 2 * (kCodes + kGroups);
};

__device__ __forceinline__ int tok(int i) { return static_cast<int>((0x67453210u >> (4 * i)) & 15u); }

// Two e4m3 scales as f16 (lo in the low half).
__device__ __forceinline__ uint32_t scales_f16x2(uint32_t lo, uint32_t hi) {
  return e4m3x2_to_f16x2(static_cast<uint16_t>(lo | (hi << 8)));
}

__device__ __forceinline__ bool is_nan_scale(uint32_t b) { return (b & 0x7fu) == 0x7fu; }

// CAUSAL: rows may see different last keys (a prefill chunk).
template <typename T, int HD, int NT, bool CAUSAL>
struct Rows {
  static constexpr bool HILO = sizeof(T) == 4;
  static constexpr int PARTS = HILO ? 2 : 1;
  static constexpr int KK = HD / 16;                    // k steps of Q K^T, m tiles of V^T P^T
  static constexpr int KD = HD / 4;                     // dims of K that a lane holds
  static constexpr int KW = KD >= 8 ? KD / 8 : 1;       // words of them
  static constexpr int DB = HD / 8;                     // dims of V^T that a lane holds
  static constexpr int VW = DB >= 8 ? DB / 8 : 1;       // words of them
  // blocks taken together, as the registers allow; a decode's, where there are many
  static constexpr int PAIR = HD * NT * PARTS <= 128 ? 2 : 1;
  static constexpr int TAKE = HD * NT * PARTS <= 64 ? 4 : PAIR;

  uint32_t qb[NT][PARTS][KK][2];
  float o[NT][KK][4];
  float m[NT][2], l[NT][2], rs[NT][2];
  int last[NT][2];
  int cut;             // least last key over the active rows
  float vg;            // the head's scale of V
  int kc, kg, vc[2], vgr[2];  // this lane's pieces: K codes and scales, V codes and scales

  // Where the lane's pieces lie in a tile.
  __device__ __forceinline__ void place() {
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    kc = tok(g) * (HD / 2) + c * KD / 2;
    kg = Tile<HD>::kKGroups + tok(g) * KK + c * KD / kGroup;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      vc[i] = Tile<HD>::kVCodes + tok(2 * c + i) * (HD / 2) + g * DB / 2;
      vgr[i] = Tile<HD>::kVGroups + tok(2 * c + i) * KK + g * DB / kGroup;
    }
  }

  // q_row(r): row r's query (null: no such row); last_key(r): the last key it sees
  // (-1: none).  factor: of a score, in log2 units; v_scale: of an output.
  template <typename QRow, typename LastKey>
  __device__ __forceinline__ void begin(QRow q_row, LastKey last_key, float factor, float v_scale) {
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    vg = v_scale;
    int least = INT_MAX;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[KK][4];
      const T* qp = q_row(nt * 8 + g);
      float a = 0.f;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        x[kk][0] = x[kk][1] = x[kk][2] = x[kk][3] = 0.f;
        if (qp) load4<T>(qp + c * KD + kk * 4, x[kk]);
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
      const float back = pow2f(-up) * factor;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = nt * 8 + 2 * c + j;
        // (not zero: a hidden key's -inf stays -inf)
        rs[nt][j] = fmaxf(__shfl_sync(0xffffffffu, back, (2 * c + j) * 4), 1.2e-38f);
        // a row without a query is never masked (and never stored)
        last[nt][j] = q_row(r) ? last_key(r) : INT_MAX;
        least = min(least, last[nt][j]);
        m[nt][j] = kNone;
        l[nt][j] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < KK; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }
    cut = __reduce_min_sync(0xffffffffu, least);
  }

  template <int W, int D>
  static __device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t (&w)[W]) {
    if constexpr (D == 32) {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else if constexpr (D == 16) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x, w[1] = x.y;
    } else if constexpr (D == 8) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (D == 4) {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
      w[0] = *p;
    }
  }

  // NB consecutive blocks: their tiles, the position j0 of the first token, the
  // sequence's tokens from there on (valid: V rows past them are not used).  Two at a
  // time share the latency of each step.  EDGE: some row may not see some of their tokens.
  template <int NB, bool EDGE>
  __device__ __forceinline__ void blocks(const uint8_t* const (&t)[NB], int j0, int valid) {
    float w[NB][NT][4];  // scores before their factor
    // ---- S^T = K Q^T
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      uint32_t kw[2][KW];
      __half2 ks[2][(KD + 15) / 16];  // [token g | g + 8]: codes; scales, twice each
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        load_codes<KW, KD>(t[nb] + kc + h * 8 * (HD / 2), kw[h]);
        const uint8_t* sp = t[nb] + kg + h * 8 * KK;
        if constexpr (KD == 32) {
          const uint32_t s2 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(sp));
          ks[h][0] = __low2half2(*reinterpret_cast<const __half2*>(&s2));
          ks[h][1] = __high2half2(*reinterpret_cast<const __half2*>(&s2));
        } else {
          const uint32_t s2 = e4m3x2_to_f16x2(*sp);
          ks[h][0] = __low2half2(*reinterpret_cast<const __half2*>(&s2));
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        w[nb][nt][0] = w[nb][nt][1] = w[nb][nt][2] = w[nb][nt][3] = 0.f;
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        uint32_t a[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          codes_to_f16x2(kw[h][i], a[h]);
          const uint32_t sc = *reinterpret_cast<const uint32_t*>(&ks[h][i / 2]);
#pragma unroll
          for (int e = 0; e < 4; ++e) a[h][e] = mul_f16x2(a[h][e], sc);
        }
#pragma unroll
        for (int e = 0; e < 2 && 2 * i + e < KK; ++e) {
          const int kk = 2 * i + e;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int pt = 0; pt < PARTS; ++pt)
              mma_f16_16816(w[nb][nt], a[0][2 * e], a[1][2 * e], a[0][2 * e + 1],
                            a[1][2 * e + 1], qb[nt][pt][kk][0], qb[nt][pt][kk][1]);
        }
      }
    }
    // ---- mask, weights
    const bool masked = EDGE && j0 + NB * kBS - 1 > cut;
    if (masked) {
      const int t0 = j0 + tok((threadIdx.x & 31) >> 2);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (t0 + nb * kBS + (e >> 1) * 8 > last[nt][e & 1]) w[nb][nt][e] = -INFINITY;
    }
    float pw[NB][NT][4];
    float add[NT][2];
    auto weigh = [&]() {  // whether some weights are past f16's range, or there is no reference
      bool past = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float cst = kWeightLog2 - m[nt][j];
          add[nt][j] = 0.f;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x = fast_exp2(fmaf(w[nb][nt][2 * e + j], rs[nt][j], cst));
              pw[nb][nt][2 * e + j] = x;
              add[nt][j] += x;
            }
          past |= add[nt][j] > kWeightMax;  // (no weight is larger than their sum)
        }
      return past;
    };
    // (without a reference m is kNone, and weights of keys that are seen come out infinite)
    if (__any_sync(0xffffffffu, weigh())) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float d[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float mx = -INFINITY;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mx = fmaxf(mx, fmaxf(w[nb][nt][j], w[nb][nt][2 + j]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float mn = fmaxf(m[nt][j], mx * rs[nt][j]);
          d[j] = fast_exp2(m[nt][j] - mn);
          m[nt][j] = mn;
          l[nt][j] *= d[j];
        }
#pragma unroll
        for (int i = 0; i < KK; ++i) {
          o[nt][i][0] *= d[0];
          o[nt][i][1] *= d[1];
          o[nt][i][2] *= d[0];
          o[nt][i][3] *= d[1];
        }
      }
      weigh();
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) l[nt][j] += add[nt][j];
    uint32_t vw[NB][4][VW];  // tokens tok(2c), tok(2c + 1), and those + 8
    uint32_t vs[NB][4];      // their scales' codes
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        load_codes<VW, DB>(t[nb] + vc[h & 1] + (h >> 1) * 8 * (HD / 2), vw[nb][h]);
        vs[nb][h] = t[nb][vgr[h & 1] + (h >> 1) * 8 * KK];
      }
    // V rows past the sequence's end hold whatever the pool holds there: codes, which
    // are finite, under scales taken as zero
    if (EDGE && valid < NB * kBS) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (nb * kBS + tok(2 * (threadIdx.x & 3) + (h & 1)) + (h >> 1) * 8 >= valid) vs[nb][h] = 0u;
    }
    bool by_term = false;
    if constexpr (CAUSAL) {
      // a NaN among the values must not reach the rows that do not see its token, as
      // it would through 0 * NaN in the product: such blocks are summed term by term
      bool nan = false;
      if (masked) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int h = 0; h < 4; ++h) nan |= is_nan_scale(vs[nb][h]);
      }
      by_term = __any_sync(0xffffffffu, nan);
    }
    // ---- O^T += V^T P^T
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if (CAUSAL && by_term) {
        add_by_term(t[nb], pw[nb], j0 + nb * kBS, valid - nb * kBS);
        continue;
      }
      uint32_t pb[NT][PARTS][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t hi = pack_f16x2(pw[nb][nt][2 * h], pw[nb][nt][2 * h + 1]);
          pb[nt][0][h] = transpose_8x8(hi);
          if constexpr (HILO) {
            const float2 f = unpack_f16x2(hi);
            pb[nt][1][h] = transpose_8x8(pack_f16x2((pw[nb][nt][2 * h] - f.x) * kLowUp,
                                                    (pw[nb][nt][2 * h + 1] - f.y) * kLowUp));
          }
        }
      const uint32_t s0 = scales_f16x2(vs[nb][0], vs[nb][1]);  // of the tokens' pairs
      const uint32_t s1 = scales_f16x2(vs[nb][2], vs[nb][3]);
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        // even and odd dims of a pair of tokens: a byte holds one dim's two codes
        uint32_t a[4][4];  // [pair 0 even, odd, pair 1 even, odd][byte]
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x = vw[nb][2 * h][i], y = vw[nb][2 * h + 1][i];
          codes_to_f16x2((x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u), a[2 * h]);
          codes_to_f16x2(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), a[2 * h + 1]);
        }
#pragma unroll
        for (int e = 0; e < 4 && 4 * i + e < KK; ++e) {
          const uint32_t a0 = mul_f16x2(a[0][e], s0), a1 = mul_f16x2(a[1][e], s0);
          const uint32_t a2 = mul_f16x2(a[2][e], s1), a3 = mul_f16x2(a[3][e], s1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (HILO) {
              float d[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16_16816(d, a0, a1, a2, a3, pb[nt][1][0], pb[nt][1][1]);
#pragma unroll
              for (int k = 0; k < 4; ++k) d[k] *= kLowDown;
              mma_f16_16816(d, a0, a1, a2, a3, pb[nt][0][0], pb[nt][0][1]);
#pragma unroll
              for (int k = 0; k < 4; ++k) o[nt][4 * i + e][k] += d[k];
            } else {
              mma_f16_16816(o[nt][4 * i + e], a0, a1, a2, a3, pb[nt][0][0], pb[nt][0][1]);
            }
          }
        }
      }
    }
  }

  // O += P V of a masked block term by term, the terms of hidden tokens left out (w is
  // 0 there but the value may be NaN).
  __device__ __forceinline__ void add_by_term(const uint8_t* t, const float (&w)[NT][4], int j0,
                                              int valid) {
    const int lane = threadIdx.x & 31;
    const int c = lane & 3;
    const int codes0 = vc[0] - tok(2 * c) * (HD / 2), groups0 = vgr[0] - tok(2 * c) * KK;
#pragma unroll 1
    for (int ti = 0; ti < kBS; ++ti) {
      const int token = tok(ti & 7) + (ti & 8);
      const float s = scale_value(t[groups0 + token * KK]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float wj = __shfl_sync(0xffffffffu, ti < 8 ? w[nt][j] : w[nt][2 + j],
                                       (ti & 7) * 4 + c);
          if (token >= valid || j0 + token > last[nt][j]) continue;
#pragma unroll
          for (int i = 0; i < KK; ++i) {
            uint32_t r[4];
            codes_to_f16x2(t[codes0 + token * (HD / 2) + i], r);
            const float2 v = unpack_f16x2(r[0]);
            o[nt][i][j] = fmaf(wj, v.x * s, o[nt][i][j]);
            o[nt][i][2 + j] = fmaf(wj, v.y * s, o[nt][i][2 + j]);
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

  // Output of every row: out_row(r) -> T* (null: skip).  A row that sees no key gets
  // zeros.
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
          x[2 * i] = o[nt][i][j] * inv * vg;
          x[2 * i + 1] = o[nt][i][2 + j] * inv * vg;
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

  // Partial result of every row: normalised output (fp32), the reference of its sum in
  // log2 units and the sum.  A NaN sum is passed on as NaN outputs with a sum of 1, so
  // that a merge that drops parts without weight keeps it.
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
          x[2 * i] = o[nt][i][j] * inv * vg;
          x[2 * i + 1] = o[nt][i][2 + j] * inv * vg;
        }
        store_f32(pp + g * DB, x);
        if (g == 0) {
          float* ml = ml_row(r);
          ml[0] = bad ? 0.f : m[nt][j];
          ml[1] = bad ? 1.f : l[nt][j];
        }
      }
  }
};

}  // namespace fp4
}  // namespace pkv
