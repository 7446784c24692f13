// What a step does to its queries, keys and values between the projection and the
// cache: the norm of each head's query and key, the rotation by position, and the
// write into a bf16 / fp32 pool or, quantised, into a 4-bit one.
//
//   z = x * rsqrt(mean(x^2) + eps) * w          (heads with a weight)
//   y = z * cos +- partner(z) * sin             (the first rot dims)
// in fp32, rounded once to the input's type; a 4-bit pool's codes are those of the
// rounded keys, so that the one call equals the two (rows out, then a write).
//
// Bound by HBM for prompts (each row is read once and written once), if what is done to
// an element stays at some six operations, and by its chain of loads (position, table
// row) for a decode step.  LPH lanes hold a head's row, 16 elements each: two vectors of
// eight whose dims turn with each other, so that a rotation needs no exchange and eight
// angles a lane.  A warp stays in one column, 32 / LPH heads of one kind (queries, keys
// or values), and goes from token to token: its kind, weights and addresses but for the
// token stay in registers (chosen anew for each token they cost as much as the
// arithmetic).  The next token's row, slot and angles, and the position after that, are
// on their way meanwhile; neighbouring warps hold the columns of one token, whose angles
// they share through L1.
//
// 8,192 tokens of 64 + 8 + 8 heads of 128, normed, turned and written, bf16: 64.7 us, 5.2
// TB/s (a copy 6.7; a warp a token instead of a column: 146).  31,722 tokens of 8 x 64
// quantised: 18.3 us, 4.6 TB/s, where issue slots are 73% taken.  A decode step of 64 tokens
// 1.9 us: the launch and that chain of loads.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "device.cuh"
#include "fp4.cuh"
#include "host_cache.h"
#include "launch.h"
#include "ragged.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Params {
  NormRopeArgs a;
  int q_cols, kv_cols;  // columns of the queries, and of the keys (values)
  int cols;             // and of all kinds
  int bs_shift;         // log2 of the block size, -1: no power of two
  float inv_hd;         // 1 / head_dim
};

enum Turn { kNoTurn, kHalves, kPairs };  // dim i with i + rot / 2; 2i with 2i + 1

// Sixteen elements of a row (two vectors of eight), as stored and as floats.
template <typename T>
struct Vec16;

template <>
struct Vec16<__nv_bfloat16> {
  uint4 w[2];
  __device__ __forceinline__ void load8(int j, const __nv_bfloat16* p) {
    w[j] = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void store8(int j, __nv_bfloat16* p) const {
    *reinterpret_cast<uint4*>(p) = w[j];
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ float amax8(int j) const { return fp4::amax8(w[j]); }
  __device__ __forceinline__ void get(float2 (&x)[8]) const {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t u[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[4 * j + i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    }
  }
  __device__ __forceinline__ void set(const float2 (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      w[j] = make_uint4(pack_bf16x2(x[4 * j].x, x[4 * j].y), pack_bf16x2(x[4 * j + 1].x, x[4 * j + 1].y),
                        pack_bf16x2(x[4 * j + 2].x, x[4 * j + 2].y),
                        pack_bf16x2(x[4 * j + 3].x, x[4 * j + 3].y));
  }
};

template <>
struct Vec16<float> {
  float4 w[4];
  __device__ __forceinline__ void load8(int j, const float* p) {
    w[2 * j] = reinterpret_cast<const float4*>(p)[0];
    w[2 * j + 1] = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store8(int j, float* p) const {
    reinterpret_cast<float4*>(p)[0] = w[2 * j];
    reinterpret_cast<float4*>(p)[1] = w[2 * j + 1];
  }
  __device__ __forceinline__ float amax8(int j) const { return fp4::amax8(w[2 * j], w[2 * j + 1]); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void get(float2 (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[2 * i] = make_float2(w[i].x, w[i].y), x[2 * i + 1] = make_float2(w[i].z, w[i].w);
  }
  __device__ __forceinline__ void set(const float2 (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = make_float4(x[2 * i].x, x[2 * i].y, x[2 * i + 1].x, x[2 * i + 1].y);
  }
};

// Sum of the squares of a row, whose LPH lanes hold x each.
template <int LPH>
__device__ __forceinline__ float sum_of_squares(const float2 (&x)[8]) {
  float2 two = __fmul2_rn(x[0], x[0]);
#pragma unroll
  for (int e = 1; e < 8; ++e) two = __ffma2_rn(x[e], x[e], two);
  float sum = two.x + two.y;
#pragma unroll
  for (int m = 1; m < LPH; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  return sum;
}

// CTAs that an SM's registers hold: a row and angles on their way and at hand, weights and
// addresses.  (With three CTAs to turn rows 30 bytes a thread spill: 8,192 tokens of 64 +
// 8 + 8 heads of 128 take 105 us in place of 65; with the angles asked for where they are
// needed 72 us, with two rows on their way 74.)
template <Turn TURN>
constexpr int kCtasPerSm = TURN == kNoTurn ? 4 : 2;

// TURN: the rotation (and norms, where there are weights); kNoTurn: rows are stored
// as they are.  FP4: the pools are 4-bit ones.
template <typename T, int LPH, Turn TURN, bool FP4>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<TURN>)
    norm_rope_kernel(const __grid_constant__ Params p) {
  const NormRopeArgs& a = p.a;
  pdl_wait();
  // (the next kernel is let in early only after a 4-bit write: a planned decode of
  // the bf16 cache reads its first K / V before it waits)
  if constexpr (TURN == kNoTurn) pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPH, l = lane % LPH;
  // ---- the warp's column, and the tokens t, t + stride, ..
  const uint32_t warp = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int stride = static_cast<int>(gridDim.x * kWarps / p.cols);
  int t = static_cast<int>(warp / p.cols);
  const int col = static_cast<int>(warp - uint32_t(t) * p.cols);
  if (t >= stride || t >= a.num_tokens) return;
  const int kind = col < p.q_cols ? 0 : col < p.q_cols + p.kv_cols ? 1 : 2;
  const int h = (kind == 0 ? col : col - p.q_cols - (kind - 1) * p.kv_cols) * (32 / LPH) + sub;
  // (head_dim / 16 need not fill the LPH lanes, nor the heads the last column)
  bool mine = l * 16 < a.head_dim && h < (kind == 0 ? a.n_heads : a.n_kv);
  // ---- the lane's two vectors: dims da .. da + 7 and db .. db + 7
  const int half = a.rot / 2;
  int da = l * 16, db = da + 8;
  const bool turns = TURN != kNoTurn && kind < 2 && l * 16 < a.rot;
  if (TURN == kHalves && l * 16 < a.rot) da = l * 8, db = da + half;
  // ---- addresses
  const int64_t pitch = kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride;
  const T* src = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + t * pitch +
                 int64_t(h) * a.head_dim;
  const bool rows_out = kind == 0 || a.slots == nullptr;
  // rows: the token's; a pool of rows: slot 0's; a 4-bit pool: the head's part of block 0
  T* dst = nullptr;
  uint8_t *codes_at = nullptr, *groups_at = nullptr;
  const int64_t out_pitch = !rows_out ? int64_t(a.n_kv) * a.head_dim
                            : kind == 0 ? a.q_out_stride : a.k_out_stride;
  float g = 1.f;
  if (rows_out) {
    dst = static_cast<T*>(kind == 0 ? a.q_out : a.k_out) + t * out_pitch + int64_t(h) * a.head_dim;
  } else if constexpr (FP4) {
    const int64_t row = int64_t(h) * a.block_size;
    codes_at = static_cast<uint8_t*>(kind == 2 ? a.v_pool : a.k_pool) + row * (a.head_dim / 2);
    groups_at = (kind == 2 ? a.v_groups : a.k_groups) + row * (a.head_dim / 16);
    if (mine) g = (kind == 2 ? a.v_scale : a.k_scale)[h];
    if (!fp4::is_head_scale(g)) {  // (its inverse would not be one: no codes for this head)
      report(a.err, PKV_DEVERR_SCALE);
      mine = false;
      g = 1.f;
    }
  } else {
    dst = static_cast<T*>(kind == 2 ? a.v_pool : a.k_pool) + int64_t(h) * a.head_dim;
  }
  // ---- what is on its way: the next token's row, slot and angles, the position after that
  const bool slots = !rows_out || (kind == 1 && a.slots != nullptr);
  Vec16<T> next;
  next.zero();
  int64_t slot_next = 0;
  auto fetch = [&]() {
    if (mine) {
      next.load8(0, src + da);
      next.load8(1, src + db);
    }
    if (slots) slot_next = a.slots[t];
  };
  fetch();
  float4 angle[4];  // cosines, then sines
  bool there_next = true;
  auto turn_to = [&](int pos) {
    there_next = pos >= 0 && pos < a.num_positions;
    if (kind == 2) return;
    // (lanes whose dims do not turn take the first ones' and leave them unused)
    const float* row = a.cos_sin + int64_t(there_next ? pos : 0) * a.rot + (turns ? l * 8 : 0);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      angle[q] = reinterpret_cast<const float4*>(row)[q];
      angle[2 + q] = reinterpret_cast<const float4*>(row + half)[q];
    }
  };
  int pos_next = 0;
  if constexpr (TURN != kNoTurn) {
    turn_to(a.positions[t]);
    if (t + stride < a.num_tokens) pos_next = a.positions[t + stride];
  }
  const T* wp = static_cast<const T*>(kind == 0 ? a.q_weight : a.k_weight);
  const bool norm = TURN != kNoTurn && kind < 2 && wp != nullptr;
  Vec16<T> weight;
  weight.zero();
  if (norm && l * 16 < a.head_dim) {
    weight.load8(0, wp + da);
    weight.load8(1, wp + db);
  }

  for (;;) {
    Vec16<T> v = next;
    const int64_t slot = slot_next;
    const bool there = there_next;
    float2 c[4], s[4];  // the lane's angles
    t += stride;
    const bool more = t < a.num_tokens;
    if (more) {
      src += stride * pitch;
      fetch();
    }
    if constexpr (TURN != kNoTurn) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        c[2 * q] = make_float2(angle[q].x, angle[q].y), c[2 * q + 1] = make_float2(angle[q].z, angle[q].w);
        s[2 * q] = make_float2(angle[2 + q].x, angle[2 + q].y);
        s[2 * q + 1] = make_float2(angle[2 + q].z, angle[2 + q].w);
      }
      if (!there && lane == 0 && col == 0) report(a.err, PKV_DEVERR_LENGTH);
      if (more) {
        turn_to(pos_next);
        if (t + stride < a.num_tokens) pos_next = a.positions[t + stride];
      }
    }

    float2 x[8];
    if (TURN != kNoTurn && kind < 2) {
      v.get(x);
      if (norm) {
        float sum = sum_of_squares<LPH>(x);
        float eps = a.eps;
        // Squares past fp32's range, or below it where no eps hides that: once more
        // with the row times a power of two.
        const bool large = !(sum <= 0x1p100f), small = sum < 0x1p-100f && eps < 0x1p-100f;
        if (__any_sync(0xffffffffu, large || small)) {
          const float m = large ? 0x1p-80f : small ? 0x1p100f : 1.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = make_float2(x[e].x * m, x[e].y * m);
          sum = sum_of_squares<LPH>(x);
          eps = eps * m * m;
        }
        const float f = rsqrtf(fmaf(sum, p.inv_hd, eps));
        const float2 f2 = make_float2(f, f);
        float2 w[8];
        weight.get(w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __fmul2_rn(__fmul2_rn(x[e], f2), w[e]);
      }
      if (turns) {
        if constexpr (TURN == kHalves) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 lo = x[e], hi = x[e + 4];
            const float2 minus = make_float2(-hi.x, -hi.y);
            x[e] = __ffma2_rn(minus, s[e], __fmul2_rn(lo, c[e]));
            x[e + 4] = __ffma2_rn(lo, s[e], __fmul2_rn(hi, c[e]));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float ce = e & 1 ? c[e / 2].y : c[e / 2].x, se = e & 1 ? s[e / 2].y : s[e / 2].x;
            const float lo = x[e].x, hi = x[e].y;
            x[e] = make_float2(fmaf(-hi, se, lo * ce), fmaf(lo, se, hi * ce));
          }
        }
      }
      if (there) v.set(x);
      else v.zero();
    }
    __syncwarp();  // (a row may be stored in place: every lane has read it by now)
    if (rows_out) {
      if (mine) {
        v.store8(0, dst + da);
        v.store8(1, dst + db);
      }
      dst += stride * out_pitch;
    } else if (static_cast<uint64_t>(slot) < static_cast<uint64_t>(a.num_slots)) {
      if (there) {
        if constexpr (FP4) {
          v.get(x);  // as rounded
          fp4::Codes codes;
          if constexpr (TURN == kHalves) {
            // the other eight elements of each vector's group lie in other lanes
            codes = fp4::quantise_apart<sizeof(T) == 4>(x, v.amax8(0), v.amax8(1), g, [&](int j, float amax_a, float amax_b) {
              const int other = ((j == 0 ? da : db) / 8) ^ 1;  // vector of the row
              const int turned = half / 8;                     // that lanes hold first
              const bool second = other < 2 * turned ? other >= turned : (other & 1);
              const int from = other < turned ? other : other < 2 * turned ? other - turned : other / 2;
              const float fa = __shfl_sync(0xffffffffu, amax_a, (sub * LPH + from) & 31);
              const float fb = __shfl_sync(0xffffffffu, amax_b, (sub * LPH + from) & 31);
              return second ? fb : fa;
            });
          } else {
            codes = fp4::quantise<sizeof(T) == 4>(x, v.amax8(0), v.amax8(1), g);
          }
          const uint32_t at = static_cast<uint32_t>(slot);  // (slots are below 2^31)
          const uint32_t blk = p.bs_shift >= 0 ? at >> p.bs_shift : at / a.block_size;
          const int64_t row = int64_t(blk) * a.n_kv * a.block_size +
                              (at - blk * static_cast<uint32_t>(a.block_size));
          if (mine) {
            uint8_t* pool = codes_at + row * (a.head_dim / 2);
            uint8_t* groups = groups_at + row * (a.head_dim / 16);
            if constexpr (TURN == kHalves) {
              *reinterpret_cast<uint32_t*>(pool + da / 2) = codes.a;
              *reinterpret_cast<uint32_t*>(pool + db / 2) = codes.b;
              if (da % 16 == 0) groups[da / 16] = static_cast<uint8_t>(codes.scale_a);
              if (db % 16 == 0) groups[db / 16] = static_cast<uint8_t>(codes.scale_b);
            } else {
              *reinterpret_cast<uint2*>(pool + da / 2) = make_uint2(codes.a, codes.b);
              groups[da / 16] = static_cast<uint8_t>(codes.scale_a);
            }
          }
        } else if (mine) {
          T* at = dst + slot * out_pitch;
          v.store8(0, at + da);
          v.store8(1, at + db);
        }
      }
    } else if (slot >= 0 && lane == 0 && kind == 1) {
      report(a.err, PKV_DEVERR_SLOT);  // (a negative slot is a padding token's)
    }
    if (!more) return;
  }
}

// One wave of CTAs at most, and columns enough for every token of a decode step.
template <typename T, int LPH, Turn TURN, bool FP4>
cudaError_t run(const Params& p, cudaStream_t stream) {
  const int64_t wave = int64_t(sm_count()) * kCtasPerSm<TURN>;
  const int64_t need = (int64_t(p.a.num_tokens) * p.cols + kWarps - 1) / kWarps;
  // (a warp for each column at the least)
  const int64_t least = (p.cols + kWarps - 1) / kWarps;
  const int64_t ctas = std::max(least, std::min(wave, need));
  return launch_pdl(norm_rope_kernel<T, LPH, TURN, FP4>, dim3(static_cast<unsigned>(ctas)),
                    kThreads, 0, stream, p);
}

template <typename T, int LPH>
cudaError_t run_turn(const Params& p, cudaStream_t stream) {
  const bool fp4 = p.a.k_groups != nullptr;
  if (p.a.cos_sin == nullptr) return run<T, LPH, kNoTurn, true>(p, stream);
  if (p.a.interleaved)
    return fp4 ? run<T, LPH, kPairs, true>(p, stream) : run<T, LPH, kPairs, false>(p, stream);
  return fp4 ? run<T, LPH, kHalves, true>(p, stream) : run<T, LPH, kHalves, false>(p, stream);
}

template <typename T>
cudaError_t run_width(const Params& p, int lph, cudaStream_t stream) {
  switch (lph) {
    case 1: return run_turn<T, 1>(p, stream);
    case 2: return run_turn<T, 2>(p, stream);
    case 4: return run_turn<T, 4>(p, stream);
    case 8: return run_turn<T, 8>(p, stream);
    default: return run_turn<T, 16>(p, stream);
  }
}

// Lanes of a head's row: the power of two that holds head_dim / 16.
int lanes_per_head(int head_dim) {
  int lph = 1;
  while (lph * 16 < head_dim) lph *= 2;
  return lph;
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  Params p{};
  p.a = a;
  const int lph = lanes_per_head(a.head_dim);
  const int rpw = 32 / lph;
  p.q_cols = (a.n_heads + rpw - 1) / rpw;
  p.kv_cols = (a.n_kv + rpw - 1) / rpw;
  p.cols = p.q_cols + p.kv_cols * (a.slots != nullptr ? 2 : 1);
  p.inv_hd = 1.f / static_cast<float>(a.head_dim);
  p.bs_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.block_size == 1 << i) p.bs_shift = i;
  return a.dtype == PKV_F32 ? run_width<float>(p, lph, stream)
                            : run_width<__nv_bfloat16>(p, lph, stream);
}

}  // namespace pkv
