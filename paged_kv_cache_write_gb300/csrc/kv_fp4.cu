// Reading a 4-bit cache back: codes and scales to contiguous rows of values.
//
// Bound by HBM: 9 / 16 byte an element in and 2 or 4 out.  A CTA reads back a
// window of 32 tokens, found by one pass over the offsets; an item is as many
// elements as fill one 16-byte store, so that a warp's stores are contiguous.  64 sequences
// of 512 - 2,048 tokens of 8 x 64 as bf16: 36.4 us, 5.7 TB/s (a copy 6.7).
#include <cuda_runtime.h>

#include <algorithm>

#include "device.cuh"
#include "fp4.cuh"
#include "host_cache.h"
#include "launch.h"
#include "ragged.cuh"

namespace pkv {

namespace {

constexpr int kThreads = kWindowThreads;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 2;   // rows a warp reads at once
constexpr int kSteps = 2;  // and steps of 32 items in each (four rows: 39 us for those 36.4)

struct GatherParams {
  const uint8_t *k_pool, *v_pool, *k_groups, *v_groups;
  const float *k_scale, *v_scale;
  const int32_t* bt;
  const int32_t* seq_lens;
  const int32_t* cu;
  uint8_t *k_out, *v_out;
  int32_t* err;
  int W, num_seqs, total, bs, num_blocks, n_kv, hd;
};

template <typename T>
struct Item;

template <>
struct Item<float> {
  using Load = uint16_t;  // 4 elements
  static __device__ __forceinline__ void store(uint8_t* dst, uint32_t u, float s) {
    uint32_t r[4];
    fp4::codes_to_f16x2(u, r);
    const float2 a = fp4::f16x2_to_float2(r[0]), b = fp4::f16x2_to_float2(r[1]);
    __stcs(reinterpret_cast<float4*>(dst), make_float4(a.x * s, a.y * s, b.x * s, b.y * s));
  }
};

template <>
struct Item<__nv_bfloat16> {
  using Load = uint32_t;  // 8 elements (their values are bf16 numbers: nothing is rounded)
  static __device__ __forceinline__ void store(uint8_t* dst, uint32_t u, float s) {
    uint32_t r[4], o[4];
    fp4::codes_to_f16x2(u, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = fp4::f16x2_to_float2(r[i]);
      o[i] = pack_bf16x2(a.x * s, a.y * s);
    }
    __stcs(reinterpret_cast<uint4*>(dst), make_uint4(o[0], o[1], o[2], o[3]));
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) kv_gather_fp4_kernel(const GatherParams p) {
  __shared__ int cnt_s[kWindow];
  __shared__ int blk_s[kWindow], off_s[kWindow];
  // The next kernel is not let in early: a planned decode of the bf16 cache reads
  // its first K / V before it waits, and these outputs may be that cache's blocks.
  pdl_wait();
  const int t0 = blockIdx.x * kWindow;
  const int n = min(kWindow, p.total - t0);
  const int b = window_seq(p.cu, p.num_seqs, t0, cnt_s);
  if (threadIdx.x < kWindow) {
    const int i = threadIdx.x;
    int blk = -1, off = 0;  // -1: nothing to read, zeros
    if (i < n) {
      if (b >= p.num_seqs) {
        report(p.err, PKV_DEVERR_LENGTH);
      } else {
        const int64_t pos = int64_t(t0) + i - p.cu[b];
        if (pos < 0 || pos >= p.seq_lens[b]) {
          report(p.err, PKV_DEVERR_LENGTH);
        } else if (pos / p.bs >= p.W) {
          report(p.err, PKV_DEVERR_TABLE_WIDTH);
        } else {
          blk = p.bt[int64_t(b) * p.W + pos / p.bs];
          off = static_cast<int>(pos % p.bs);
          if (blk < 0 || blk >= p.num_blocks) {
            report(p.err, PKV_DEVERR_BLOCK_ID);
            blk = -1;
          }
        }
      }
    }
    blk_s[i] = blk;
    off_s[i] = off;
  }
  __syncthreads();
  using Load = typename Item<T>::Load;
  constexpr int E = 2 * sizeof(Load);  // elements per item
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int iph = p.hd / E;       // items of a head
  const int ipr = p.n_kv * iph;   // and of a row
  const bool pow2 = (iph & (iph - 1)) == 0;
  const int shift = 31 - __clz(iph);
  const int64_t head_step = int64_t(p.bs) * p.hd;  // elements from a block's head to its next
  // rows 0 .. n - 1 are K's, n .. 2 n - 1 V's
  for (int r0 = (blockIdx.y * kWarps + warp) * kRows; r0 < 2 * n; r0 += gridDim.y * kWarps * kRows) {
    const uint8_t *src[kRows], *grp[kRows];
    const float* scale[kRows];
    uint8_t* dst[kRows];
    bool have[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int r = min(r0 + k, 2 * n - 1);  // past the last row: it again
      const bool is_v = r >= n;
      const int t = is_v ? r - n : r;
      have[k] = blk_s[t] >= 0;
      const int64_t row = int64_t(max(blk_s[t], 0)) * p.n_kv * p.bs + off_s[t];  // of head 0
      src[k] = (is_v ? p.v_pool : p.k_pool) + row * (p.hd / 2);
      grp[k] = (is_v ? p.v_groups : p.k_groups) + row * (p.hd / 16);
      scale[k] = is_v ? p.v_scale : p.k_scale;
      dst[k] = (is_v ? p.v_out : p.k_out) + int64_t(t0 + t) * ipr * 16;
    }
    for (int c0 = lane; c0 < ipr; c0 += 32 * kSteps) {
      Load w[kRows][kSteps];
      uint8_t g[kRows][kSteps];
      float s[kRows][kSteps];
#pragma unroll
      for (int q = 0; q < kSteps; ++q) {
        const int c = min(c0 + 32 * q, ipr - 1);
        const int h = pow2 ? c >> shift : c / iph;
        const int i = c - h * iph;  // item of the head
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
          w[k][q] = __ldcs(reinterpret_cast<const Load*>(src[k] + h * (head_step / 2)) + i);
          g[k][q] = grp[k][h * (head_step / 16) + i * E / fp4::kGroup];
          s[k][q] = scale[k][h];
        }
      }
#pragma unroll
      for (int q = 0; q < kSteps; ++q) {
        const int c = c0 + 32 * q;
        if (c < ipr) {
#pragma unroll
          for (int k = 0; k < kRows; ++k)
            if (r0 + k < 2 * n)
              Item<T>::store(dst[k] + int64_t(c) * 16, have[k] ? w[k][q] : 0u,
                             have[k] ? fp4::scale_value(g[k][q]) * s[k][q] : 0.f);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_gather_fp4(const Fp4Cache& c, const PoolShape& pool, const int32_t* bt,
                                 int32_t W, const int32_t* seq_lens, const int32_t* cu,
                                 int32_t num_seqs, int32_t total_tokens, int32_t dtype,
                                 void* k_out, void* v_out, int32_t* err, cudaStream_t stream) {
  if (total_tokens == 0) return cudaSuccess;
  GatherParams p{};
  p.k_pool = static_cast<const uint8_t*>(c.k_pool);
  p.v_pool = static_cast<const uint8_t*>(c.v_pool);
  p.k_groups = static_cast<const uint8_t*>(c.k_groups);
  p.v_groups = static_cast<const uint8_t*>(c.v_groups);
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
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
  // (few windows: each over several CTAs, so that a warp has one step)
  const int64_t windows = (int64_t(total_tokens) + kWindow - 1) / kWindow;
  const int64_t most = 2 * kWindow / (kWarps * kRows);
  const dim3 grid(static_cast<unsigned>(windows),
                  static_cast<unsigned>(std::max<int64_t>(1, std::min(most, sm_count() / windows))));
  return launch_pdl(dtype == PKV_F32 ? kv_gather_fp4_kernel<float>
                                     : kv_gather_fp4_kernel<__nv_bfloat16>,
                    grid, kThreads, 0, stream, p);
}

}  // namespace pkv
