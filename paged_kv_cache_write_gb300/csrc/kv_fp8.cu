// The 8-bit cache: quantise K/V as they are written, and read them back.
//
// Write.  A unit is (sequence, block that its new tokens touch, KV head, K or
// V).  With a = max |x| over the unit's new elements, its scale becomes
//   s = 2^e(a)              if the block's first token is among the new ones,
//   s = max(s_old, 2^e(a))  if the block holds earlier tokens,
// every new element is stored as e4m3(x / s), and if s grew the earlier rows'
// bytes become e4m3(value * s_old / s).  One warp holds a whole unit (16
// tokens x 128 elements of bf16 are 32 registers a lane), so K/V are read
// once, the maximum is one warp reduction and nothing leaves the SM between.
//
// Both kernels move each byte once and do next to nothing with it: they are
// bound by HBM for prompts and by their chain of dependent loads (offsets,
// length, table entry, row) for a decode step.
#include <cuda_runtime.h>

#include <algorithm>

#include "device.cuh"
#include "fp8.cuh"
#include "host_cache.h"
#include "launch.h"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kWindow = 16;  // consecutive tokens whose runs one CTA column handles
constexpr int kHeld = 8;     // 8-element vectors of a unit a lane holds

// Sequences of the tokens t0 .. t0 + n - 1 (n <= 32) of a ragged batch, by
// the whole CTA: seq_s[i] = number of sequences that end at or before token
// t0 + i, i.e. its sequence (num_seqs if it lies past the last).  One pass
// over the offsets with every load in flight, not a chain of dependent ones.
__device__ __forceinline__ void window_seqs(const int32_t* __restrict__ cu, int num_seqs, int t0,
                                            int n, int* cnt_s, int* seq_s) {
  const int tid = threadIdx.x;
  if (tid <= n) cnt_s[tid] = 0;  // [0]: ends at or before t0; [i]: ends at t0 + i
  __syncthreads();
  int before = 0;
#pragma unroll 4
  for (int i = tid; i < num_seqs; i += kThreads) {
    const int end = __ldg(cu + i + 1);
    if (end <= t0) ++before;
    else if (end < t0 + n) atomicAdd(cnt_s + (end - t0), 1);
  }
  before = __reduce_add_sync(0xffffffffu, before);
  if ((tid & 31) == 0 && before > 0) atomicAdd(cnt_s, before);
  __syncthreads();
  if (tid < 32) {
    int x = tid < n ? cnt_s[tid] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (tid >= o) x += y;
    }
    if (tid < n) seq_s[tid] = x;
  }
}

struct WriteParams {
  const uint8_t *k, *v;  // new rows
  uint8_t *k_pool, *v_pool;
  float *k_scales, *v_scales;
  const int32_t* bt;
  const int32_t* seq_lens;
  const int32_t* cu;
  int32_t* err;
  int W, num_seqs, num_tokens, bs, num_blocks, n_kv, hd;
};

// Eight consecutive elements of a row as loaded.
template <typename T>
struct Vec8;

template <>
struct Vec8<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const uint8_t* p) {
    w = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ float2 pair(int i) const {
    const uint32_t u = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
};

template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const uint8_t* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float2 pair(int i) const {
    return i == 0 ? make_float2(a.x, a.y) : i == 1 ? make_float2(a.z, a.w)
         : i == 2 ? make_float2(b.x, b.y) : make_float2(b.z, b.w);
  }
};

// max(a, |x|) over the vector; fmaxf passes over NaN.
template <typename T>
__device__ __forceinline__ float vec_amax(const Vec8<T>& v, float a) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = v.pair(i);
    a = fmaxf(a, fmaxf(fabsf(x.x), fabsf(x.y)));
  }
  return a;
}

// VPR: 8-element vectors of a head's row (0: read from p.hd).
template <typename T, int VPR>
__global__ void __launch_bounds__(kThreads) kv_write_fp8_kernel(const WriteParams p) {
  __shared__ int cnt_s[33], seq_s[32];
  __shared__ int4 run_s[kWindow];  // first token, tokens, offset in the block, block
  __shared__ int runs_s;
  const int t0 = blockIdx.x * kWindow;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  window_seqs(p.cu, p.num_seqs, t0, kWindow, cnt_s, seq_s);
  if (warp == 0) {
    __syncwarp();
    // a run: the new tokens of one sequence in one block.  Lane i looks at
    // token t0 + i: it begins a run if it is its sequence's first new token
    // or the first of a block.
    const int t = t0 + lane;
    int4 run = make_int4(0, 0, 0, 0);
    bool begins = false;
    if (lane < kWindow && t < p.num_tokens) {
      const int b = seq_s[lane];
      if (b >= p.num_seqs) {
        report(p.err, PKV_DEVERR_LENGTH);  // offsets that stop short of the token count
      } else {
        const int start = __ldg(p.cu + b), end = __ldg(p.cu + b + 1);
        const int L = __ldg(p.seq_lens + b);
        const int64_t pos = int64_t(L) - end + t;
        if (L < 0 || start < 0 || end - start > L || end > p.num_tokens || pos < 0) {
          report(p.err, PKV_DEVERR_LENGTH);
        } else if (pos / p.bs >= p.W) {
          report(p.err, PKV_DEVERR_TABLE_WIDTH);
        } else {
          const int off = static_cast<int>(pos % p.bs);
          begins = t == start || off == 0;
          if (begins) {
            const int blk = __ldg(p.bt + int64_t(b) * p.W + pos / p.bs);
            if (blk < 0 || blk >= p.num_blocks) {
              report(p.err, PKV_DEVERR_BLOCK_ID);
              begins = false;
            }
            run = make_int4(t, min(p.bs - off, end - t), off, blk);
          }
        }
      }
    }
    const unsigned m = __ballot_sync(0xffffffffu, begins);
    if (begins) run_s[__popc(m & ((1u << lane) - 1u))] = run;
    if (lane == 0) runs_s = __popc(m);
  }
  __syncthreads();

  const int vpr = VPR > 0 ? VPR : p.hd / 8;
  const int units = runs_s * 2 * p.n_kv;
  const int64_t src_row = int64_t(p.n_kv) * p.hd * sizeof(T);
  const int64_t dst_row = int64_t(p.n_kv) * p.hd;
  for (int u = blockIdx.y * kWarps + warp; u < units; u += gridDim.y * kWarps) {
    const int ri = u / (2 * p.n_kv);
    const int rem = u - ri * 2 * p.n_kv;
    const bool is_v = rem >= p.n_kv;
    const int h = is_v ? rem - p.n_kv : rem;
    const int4 run = run_s[ri];
    const int off = run.z;
    float* scale = (is_v ? p.v_scales : p.k_scales) + int64_t(run.w) * p.n_kv + h;
    const float old = off > 0 ? *scale : 0.f;
    const uint8_t* src = (is_v ? p.v : p.k) + (int64_t(run.x) * p.n_kv + h) * p.hd * sizeof(T);
    // row 0 of the block
    uint8_t* dst = (is_v ? p.v_pool : p.k_pool) + (int64_t(run.w) * p.bs * p.n_kv + h) * p.hd;
    const int nv = run.y * vpr;
    Vec8<T> v[kHeld];
    auto load = [&](int base) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int e = base + i * 32 + lane;
        if (e < nv) {
          const int r = e / vpr;
          v[i].load(src + r * src_row + (e - r * vpr) * 8 * sizeof(T));
        } else {
          v[i].zero();
        }
      }
    };
    float a = 0.f;
    for (int base = 0; base < nv; base += kHeld * 32) {
      load(base);
#pragma unroll
      for (int i = 0; i < kHeld; ++i) a = vec_amax<T>(v[i], a);
    }
    // non-negative floats order as their bits
    a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
    const float fit = fp8_scale_for(a);
    const float s = off > 0 ? fmaxf(old, fit) : fit;
    const float inv = 1.f / s;  // exact: s is a power of two
    for (int base = 0; base < nv; base += kHeld * 32) {
      if (nv > kHeld * 32) load(base);  // a unit too large to hold: read again
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int e = base + i * 32 + lane;
        if (e < nv) {
          uint32_t q[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = v[i].pair(j);
            q[j] = e4m3x2(f.x * inv, f.y * inv);
          }
          const int r = e / vpr;
          *reinterpret_cast<uint2*>(dst + (off + r) * dst_row + (e - r * vpr) * 8) =
              make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
        }
      }
    }
    if (off > 0 && s != old) {  // the scale grew: the earlier rows move to it
      const float ratio = old * inv;
      for (int e = lane; e < off * vpr; e += 32) {
        const int r = e / vpr;
        uint2* at = reinterpret_cast<uint2*>(dst + r * dst_row + (e - r * vpr) * 8);
        const uint2 w = *at;
        auto moved = [&](uint32_t u4) {
          const float2 lo = e4m3x2_to_float2(static_cast<uint16_t>(u4));
          const float2 hi = e4m3x2_to_float2(static_cast<uint16_t>(u4 >> 16));
          return e4m3x2(lo.x * ratio, lo.y * ratio) | (e4m3x2(hi.x * ratio, hi.y * ratio) << 16);
        };
        *at = make_uint2(moved(w.x), moved(w.y));
      }
    }
    if (lane == 0 && (off == 0 || s != old)) *scale = s;
  }
}

// ------------------------------------------------------------------ gather

constexpr int kGatherTokens = 32;
constexpr int kGatherUnroll = 4;

struct GatherParams {
  const uint8_t *k_pool, *v_pool;
  const float *k_scales, *v_scales;
  const int32_t* bt;
  const int32_t* seq_lens;
  const int32_t* cu;
  uint8_t *k_out, *v_out;
  int32_t* err;
  int W, num_seqs, total, bs, num_blocks, n_kv, hd;
};

// 16 values of the cache in the output type (exact in both).
template <typename T>
__device__ __forceinline__ void store16(uint8_t* dst, const uint4& w, float s);

template <>
__device__ __forceinline__ void store16<float>(uint8_t* dst, const uint4& w, float s) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = e4m3x2_to_float2(static_cast<uint16_t>(u[i]));
    const float2 b = e4m3x2_to_float2(static_cast<uint16_t>(u[i] >> 16));
    __stcs(reinterpret_cast<float4*>(dst) + i, make_float4(a.x * s, a.y * s, b.x * s, b.y * s));
  }
}

template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(uint8_t* dst, const uint4& w, float s) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 a = e4m3x2_to_float2(static_cast<uint16_t>(u[2 * i + j]));
      const float2 b = e4m3x2_to_float2(static_cast<uint16_t>(u[2 * i + j] >> 16));
      o[2 * j] = pack_bf16x2(a.x * s, a.y * s);
      o[2 * j + 1] = pack_bf16x2(b.x * s, b.y * s);
    }
    __stcs(reinterpret_cast<uint4*>(dst) + i, make_uint4(o[0], o[1], o[2], o[3]));
  }
}

// A CTA reads back kGatherTokens rows of K and of V; a thread handles 16
// elements (one 16-byte load) at a time, kGatherUnroll loads in flight.
template <typename T>
__global__ void __launch_bounds__(kThreads) kv_gather_fp8_kernel(const GatherParams p) {
  __shared__ int cnt_s[33], seq_s[32];
  __shared__ int blk_s[kGatherTokens], off_s[kGatherTokens];
  const int t0 = blockIdx.x * kGatherTokens;
  const int n = min(kGatherTokens, p.total - t0);
  window_seqs(p.cu, p.num_seqs, t0, kGatherTokens, cnt_s, seq_s);
  if (threadIdx.x < 32) {
    __syncwarp();
    const int i = threadIdx.x;
    int blk = -1, off = 0;  // -1: nothing to read, zeros
    if (i < n) {
      const int b = seq_s[i];
      if (b >= p.num_seqs) {
        report(p.err, PKV_DEVERR_LENGTH);
      } else {
        const int pos = t0 + i - __ldg(p.cu + b);
        if (pos < 0 || pos >= __ldg(p.seq_lens + b)) {
          report(p.err, PKV_DEVERR_LENGTH);
        } else if (pos / p.bs >= p.W) {
          report(p.err, PKV_DEVERR_TABLE_WIDTH);
        } else {
          blk = __ldg(p.bt + int64_t(b) * p.W + pos / p.bs);
          off = pos % p.bs;
          if (blk < 0 || blk >= p.num_blocks) {
            report(p.err, PKV_DEVERR_BLOCK_ID);
            blk = -1;
          }
        }
      }
      blk_s[i] = blk;
      off_s[i] = off;
    }
  }
  __syncthreads();
  const int wpr = p.n_kv * p.hd / 16;  // 16-element words of a row
  const int wph = p.hd / 16;
  const int items = 2 * n * wpr;
  for (int i0 = threadIdx.x; i0 < items; i0 += kThreads * kGatherUnroll) {
    uint4 w[kGatherUnroll];
    float s[kGatherUnroll];
#pragma unroll
    for (int k = 0; k < kGatherUnroll; ++k) {
      const int i = i0 + k * kThreads;
      w[k] = make_uint4(0u, 0u, 0u, 0u);
      s[k] = 0.f;
      if (i >= items) continue;
      const bool is_v = i >= n * wpr;
      const int j = is_v ? i - n * wpr : i;
      const int t = j / wpr, c = j - t * wpr;
      const int blk = blk_s[t];
      if (blk < 0) continue;
      w[k] = __ldcs(reinterpret_cast<const uint4*>(is_v ? p.v_pool : p.k_pool) +
                    (int64_t(blk) * p.bs + off_s[t]) * wpr + c);
      s[k] = __ldg((is_v ? p.v_scales : p.k_scales) + int64_t(blk) * p.n_kv + c / wph);
    }
#pragma unroll
    for (int k = 0; k < kGatherUnroll; ++k) {
      const int i = i0 + k * kThreads;
      if (i >= items) continue;
      const bool is_v = i >= n * wpr;
      const int j = is_v ? i - n * wpr : i;
      store16<T>((is_v ? p.v_out : p.k_out) + (int64_t(t0) * wpr + j) * 16 * sizeof(T), w[k], s[k]);
    }
  }
}

}  // namespace

template <typename T>
static cudaError_t write_as(const WriteParams& p, dim3 grid, cudaStream_t stream) {
  switch (p.hd) {
    case 16: kv_write_fp8_kernel<T, 2><<<grid, kThreads, 0, stream>>>(p); break;
    case 32: kv_write_fp8_kernel<T, 4><<<grid, kThreads, 0, stream>>>(p); break;
    case 64: kv_write_fp8_kernel<T, 8><<<grid, kThreads, 0, stream>>>(p); break;
    case 128: kv_write_fp8_kernel<T, 16><<<grid, kThreads, 0, stream>>>(p); break;
    default: kv_write_fp8_kernel<T, 0><<<grid, kThreads, 0, stream>>>(p); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_kv_write_fp8(const void* k, const void* v, int32_t dtype, const int32_t* bt,
                                int32_t W, const int32_t* seq_lens, const int32_t* cu,
                                int32_t num_seqs, int32_t num_tokens, void* k_pool, void* v_pool,
                                float* k_scales, float* v_scales, const PoolShape& pool,
                                int32_t* err, cudaStream_t stream) {
  if (num_tokens == 0) return cudaSuccess;
  WriteParams p{};
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.k_pool = static_cast<uint8_t*>(k_pool);
  p.v_pool = static_cast<uint8_t*>(v_pool);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.bt = bt;
  p.seq_lens = seq_lens;
  p.cu = cu;
  p.err = err;
  p.W = W;
  p.num_seqs = num_seqs;
  p.num_tokens = num_tokens;
  p.bs = pool.block_size;
  p.num_blocks = pool.num_blocks;
  p.n_kv = pool.n_kv;
  p.hd = pool.head_dim;
  // enough warps per window that each has about one unit: a window of 16
  // tokens holds about 16 / block_size + 16 * num_seqs / num_tokens runs
  const int64_t runs = std::min<int64_t>(
      std::min(kWindow, num_tokens),
      kWindow / pool.block_size + 1 + int64_t(kWindow) * num_seqs / num_tokens);
  const int64_t per = (runs * 2 * pool.n_kv + kWarps - 1) / kWarps;
  const dim3 grid(static_cast<unsigned>((int64_t(num_tokens) + kWindow - 1) / kWindow),
                  static_cast<unsigned>(std::min<int64_t>(per, 1024)));
  return dtype == PKV_F32 ? write_as<float>(p, grid, stream)
                          : write_as<__nv_bfloat16>(p, grid, stream);
}

cudaError_t launch_kv_gather_fp8(const void* k_pool, const void* v_pool, const float* k_scales,
                                 const float* v_scales, const PoolShape& pool, const int32_t* bt,
                                 int32_t W, const int32_t* seq_lens, const int32_t* cu,
                                 int32_t num_seqs, int32_t total_tokens, int32_t dtype,
                                 void* k_out, void* v_out, int32_t* err, cudaStream_t stream) {
  if (total_tokens == 0) return cudaSuccess;
  GatherParams p{};
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.bt = bt;
  p.seq_lens = seq_lens;
  p.cu = cu;
  p.k_out = static_cast<uint8_t*>(k_out);
  p.v_out = static_cast<uint8_t*>(v_out);
  p.err = err;
  p.W = W;
  p.num_seqs = num_seqs;
  p.total = total_tokens;
  p.bs = pool.block_size;
  p.num_blocks = pool.num_blocks;
  p.n_kv = pool.n_kv;
  p.hd = pool.head_dim;
  const unsigned grid = static_cast<unsigned>((int64_t(total_tokens) + kGatherTokens - 1) /
                                              kGatherTokens);
  if (dtype == PKV_F32)
    kv_gather_fp8_kernel<float><<<grid, kThreads, 0, stream>>>(p);
  else
    kv_gather_fp8_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace pkv
