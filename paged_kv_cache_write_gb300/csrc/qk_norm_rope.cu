// What a step does to its queries, keys and values between the projection and the
// cache: the norm of each head's query and key, the rotation by position, and the
// write into a bf16 / fp32 pool or, quantised, into a 4-bit one.
//
//   z = x * rsqrt(mean(x^2) + eps) * w          (heads with a weight)
//   y = z * cos +- partner(z) * sin             (the first rot dims)
// in fp32, rounded once to the input's type; a 4-bit pool's codes are those of the
// rounded keys, so that the one call equals the two (rows out, then a write).
//
// Bound by HBM for prompts (each row is read once and written once; it takes some
// 12 operations an element) and by its chain of loads (position, table row and
// row) for a decode step.  LPH lanes hold a head's row, 16 elements each: that is
// a group of the 4-bit cache, so a group's maximum needs no exchange, and the
// rotation's other halves come as a second load of the same lines (L1) rather than
// as 16 shuffles.  The angles of a lane's dims are the same for every head, and
// stay in registers while a warp goes through some of a token's rows.
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
  int rows;   // rows of a token: query heads, key heads and, where they are stored, value heads
  int passes; // rows that a warp does one after the other
  int tasks;  // warps per token
  int total;  // and of the call
};

// Sixteen consecutive elements of a row, as stored and as floats.
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
  __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t u[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[8 * j + 2 * i] = __uint_as_float(u[i] << 16);
        x[8 * j + 2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void set(const float (&x)[16]) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      w[j] = make_uint4(pack_bf16x2(x[8 * j], x[8 * j + 1]), pack_bf16x2(x[8 * j + 2], x[8 * j + 3]),
                        pack_bf16x2(x[8 * j + 4], x[8 * j + 5]),
                        pack_bf16x2(x[8 * j + 6], x[8 * j + 7]));
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
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[4 * i] = w[i].x, x[4 * i + 1] = w[i].y, x[4 * i + 2] = w[i].z, x[4 * i + 3] = w[i].w;
  }
  __device__ __forceinline__ void set(const float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
};

// Sum of the squares of a row, whose LPH lanes hold x each.
template <int LPH>
__device__ __forceinline__ float sum_of_squares(const float (&x)[16]) {
  float sum = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
  for (int m = 1; m < LPH; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  return sum;
}

// TURN: norm and rotation (else rows are stored as they are).  FP4: the pools are
// 4-bit ones.  A warp's task: some rows of one token, 32 / LPH at a time.
template <typename T, int LPH, bool TURN, bool FP4>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const Params p) {
  const NormRopeArgs& a = p.a;
  pdl_wait();
  // (the next kernel is let in early only after a 4-bit write: a planned decode of
  // the bf16 cache reads its first K / V before it waits)
  if constexpr (!TURN && FP4) pdl_launch_dependents();
  constexpr int RPW = 32 / LPH;
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPH, d0 = (lane % LPH) * 16;
  const int task = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (task >= p.total) return;
  const int t = task / p.tasks;
  const int r0 = (task - t * p.tasks) * p.passes * RPW;
  const bool has = d0 < a.head_dim;  // (head_dim / 16 need not fill the LPH lanes)

  // ---- where the token's keys and values go
  int64_t slot = 0;
  bool keep = true;
  if (a.slots != nullptr) {
    slot = a.slots[t];
    keep = slot >= 0 && slot < a.num_slots;
    if (slot >= a.num_slots && lane == 0 && r0 == 0) report(a.err, PKV_DEVERR_SLOT);
  }
  // ---- the lane's angles: y = z c + other(z) s
  float c[16], s[16];
  int other[2] = {-1, -1};  // first element of the 8 that vector j turns with (-1: none)
  bool there = true;
  if constexpr (TURN) {
    const int pos = a.positions[t];
    there = pos >= 0 && pos < a.num_positions;
    if (!there && lane == 0 && r0 == 0) report(a.err, PKV_DEVERR_LENGTH);
    const float* row = a.cos_sin + int64_t(there ? pos : 0) * a.rot;
    const int half = a.rot / 2;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int d = d0 + 8 * j;
#pragma unroll
      for (int e = 0; e < 8; ++e) c[8 * j + e] = 1.f, s[8 * j + e] = 0.f;
      if (d < a.rot && has) {
        if (a.interleaved) {
          const float4 cv = *reinterpret_cast<const float4*>(row + d / 2);
          const float4 sv = *reinterpret_cast<const float4*>(row + half + d / 2);
          const float ca[4] = {cv.x, cv.y, cv.z, cv.w}, sa[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            c[8 * j + e] = ca[e / 2];
            s[8 * j + e] = (e & 1) ? sa[e / 2] : -sa[e / 2];
          }
        } else {
          const bool low = d < half;
          const int i = low ? d : d - half;
          other[j] = low ? d + half : i;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float4 cv = reinterpret_cast<const float4*>(row + i)[q];
            const float4 sv = reinterpret_cast<const float4*>(row + half + i)[q];
            const float ca[4] = {cv.x, cv.y, cv.z, cv.w}, sa[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              c[8 * j + 4 * q + e] = ca[e];
              s[8 * j + 4 * q + e] = low ? -sa[e] : sa[e];
            }
          }
        }
      }
    }
  }

  for (int i = 0; i < p.passes; ++i) {
    const int r = r0 + i * RPW + sub;
    const bool is_q = r < a.n_heads;
    const bool is_v = r >= a.n_heads + a.n_kv;
    const int h = is_q ? r : is_v ? r - a.n_heads - a.n_kv : r - a.n_heads;  // head of its kind
    const bool mine = r < p.rows && has;
    const T* src = static_cast<const T*>(is_q ? a.q : is_v ? a.v : a.k) +
                   int64_t(t) * (is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride) +
                   int64_t(h) * a.head_dim;
    Vec16<T> v;
    v.zero();
    if (mine) {
      v.load8(0, src + d0);
      v.load8(1, src + d0 + 8);
    }
    float x[16];
    if constexpr (TURN) {
      Vec16<T> o;
      o.zero();
      const bool turns = mine && !is_v;
      if (turns && other[0] >= 0) o.load8(0, src + other[0]);
      if (turns && other[1] >= 0) o.load8(1, src + other[1]);
      __syncwarp();  // (a row may be stored in place: every lane has read it by now)
      v.get(x);
      float z[16];  // what each element turns with
      o.get(z);
      const T* w = static_cast<const T*>(is_q ? a.q_weight : a.k_weight);
      if (a.q_weight != nullptr || a.k_weight != nullptr) {
        float sum = sum_of_squares<LPH>(x);
        float eps = a.eps;
        // Squares past fp32's range, or below it where no eps hides that: once more
        // with the row times a power of two.
        const bool large = !(sum <= 0x1p100f), small = sum < 0x1p-100f && eps < 0x1p-100f;
        if (__any_sync(0xffffffffu, large || small)) {
          const float u = large ? 0x1p-80f : small ? 0x1p100f : 1.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (turns && w != nullptr) x[e] *= u, z[e] *= u;
          }
          sum = sum_of_squares<LPH>(x);
          eps = eps * u * u;
        }
        if (turns && w != nullptr) {
          const float f = rsqrtf(sum / static_cast<float>(a.head_dim) + eps);
          Vec16<T> wv;
          float wx[16];
          wv.load8(0, w + d0);
          wv.load8(1, w + d0 + 8);
          wv.get(wx);
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = x[e] * f * wx[e];
          wv.zero();
          if (other[0] >= 0) wv.load8(0, w + other[0]);
          if (other[1] >= 0) wv.load8(1, w + other[1]);
          wv.get(wx);
#pragma unroll
          for (int e = 0; e < 16; ++e) z[e] = z[e] * f * wx[e];
        }
      }
      if (a.interleaved) {
        // (a pair that does not turn has s = 0, and no part in the other: 0 x Inf)
#pragma unroll
        for (int e = 0; e < 16; ++e) z[e] = s[e] == 0.f ? 0.f : x[e ^ 1];
      }
      if (turns) {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = fmaf(x[e], c[e], z[e] * s[e]);
        if (!there) {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = 0.f;
        }
        v.set(x);
      }
    }
    if (!mine) continue;
    if (is_q || a.slots == nullptr) {
      T* dst = static_cast<T*>(is_q ? a.q_out : a.k_out) +
               int64_t(t) * (is_q ? a.q_out_stride : a.k_out_stride) + int64_t(h) * a.head_dim;
      v.store8(0, dst + d0);
      v.store8(1, dst + d0 + 8);
    } else if (keep && there) {
      if constexpr (FP4) {
        v.get(x);  // as rounded
        uint2 codes;
        uint32_t scale;
        fp4::quantise<sizeof(T) == 4>(x, 1.f / (is_v ? a.v_scale : a.k_scale)[h], codes, scale);
        const int64_t blk = slot / a.block_size;
        const int64_t row = (blk * a.n_kv + h) * a.block_size + (slot - blk * a.block_size);
        uint8_t* pool = static_cast<uint8_t*>(is_v ? a.v_pool : a.k_pool);
        *reinterpret_cast<uint2*>(pool + row * (a.head_dim / 2) + d0 / 2) = codes;
        (is_v ? a.v_groups : a.k_groups)[row * (a.head_dim / 16) + d0 / 16] =
            static_cast<uint8_t>(scale);
      } else {
        T* dst = static_cast<T*>(is_v ? a.v_pool : a.k_pool) +
                 (slot * a.n_kv + h) * a.head_dim;
        v.store8(0, dst + d0);
        v.store8(1, dst + d0 + 8);
      }
    }
  }
}

template <typename T, int LPH>
cudaError_t run(const Params& p, unsigned grid, bool fp4, cudaStream_t stream) {
  if (p.a.cos_sin == nullptr)
    return launch_pdl(norm_rope_kernel<T, LPH, false, true>, dim3(grid), kThreads, 0, stream, p);
  if (fp4)
    return launch_pdl(norm_rope_kernel<T, LPH, true, true>, dim3(grid), kThreads, 0, stream, p);
  return launch_pdl(norm_rope_kernel<T, LPH, true, false>, dim3(grid), kThreads, 0, stream, p);
}

template <typename T>
cudaError_t run_width(const Params& p, int lph, unsigned grid, bool fp4, cudaStream_t stream) {
  switch (lph) {
    case 1: return run<T, 1>(p, grid, fp4, stream);
    case 2: return run<T, 2>(p, grid, fp4, stream);
    case 4: return run<T, 4>(p, grid, fp4, stream);
    case 8: return run<T, 8>(p, grid, fp4, stream);
    default: return run<T, 16>(p, grid, fp4, stream);
  }
}

// Lanes of a head's row: the power of two that holds head_dim / 16.
int lanes_per_head(int head_dim) {
  int lph = 1;
  while (lph * 16 < head_dim) lph *= 2;
  return lph;
}

}  // namespace

int64_t norm_rope_max_tokens(int32_t rows, int32_t head_dim) {
  const int rpw = 32 / lanes_per_head(head_dim);
  return (int64_t(INT_MAX) - kWarps) / ((int64_t(rows) + rpw - 1) / rpw);
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  Params p{};
  p.a = a;
  p.rows = a.n_heads + a.n_kv * (a.slots != nullptr ? 2 : 1);
  const int lph = lanes_per_head(a.head_dim);
  const int rpw = 32 / lph;
  const int steps = (p.rows + rpw - 1) / rpw;  // of a token
  // A decode step's warps take one step each; where there are warps enough for
  // every SM several times over, one goes through more of a token's rows.
  const int64_t all = int64_t(a.num_tokens) * steps;
  const int64_t fill = int64_t(sm_count()) * 64;
  p.passes = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(steps, all / fill)));
  p.tasks = (steps + p.passes - 1) / p.passes;
  p.total = a.num_tokens * p.tasks;
  const unsigned grid = static_cast<unsigned>((int64_t(p.total) + kWarps - 1) / kWarps);
  const bool fp4 = a.k_groups != nullptr;
  return a.dtype == PKV_F32 ? run_width<float>(p, lph, grid, fp4, stream)
                            : run_width<__nv_bfloat16>(p, lph, grid, fp4, stream);
}

}  // namespace pkv
