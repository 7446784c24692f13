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
// length, table entry, row) for a decode step.  Measured, where a plain copy
// reaches 6.79 TB/s: writing 64 prompts of 1,000 - 2,000 tokens of 8 x 128 bf16
// 89 us (6.6 TB/s), of 8 x 64 56 us (5.3), 31,722 tokens of 8 x 64 23 us (4.2:
// start and last CTAs show; at 64 registers the bf16 kernels of heads of 16 - 64,
// two units at a time, spill 48 bytes a thread), reading back 64 sequences of 512 -
// 2,048 tokens of 8 x 64 39 us (6.2 TB/s; in fp32 66 us, 6.1), a decode step's
// write or a toy read-back 3.3 - 3.7 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "device.cuh"
#include "fp8.cuh"
#include "host_cache.h"
#include "launch.h"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kWindow = 32;  // consecutive tokens that one CTA (column) handles: a warp's lanes
constexpr int kHeld = 8;     // 8-element vectors that a lane holds

// Sequences of the window's tokens of a ragged batch, by the whole CTA: lane i of
// warp 0 gets the number of sequences that end at or before token t0 + i, i.e. its
// sequence (num_seqs if it lies past the last).  One pass over the offsets with
// every load in flight, not a chain of dependent ones.
__device__ __forceinline__ int window_seq(const int32_t* cu, int num_seqs, int t0, int* cnt_s) {
  const int tid = threadIdx.x;
  if (tid < kWindow) cnt_s[tid] = 0;  // [0]: ends at or before t0; [i]: ends at t0 + i
  __syncthreads();
  const int t1 = t0 + min(kWindow, INT_MAX - t0);
  int before = 0;
#pragma unroll 4
  for (int i = tid; i < num_seqs; i += kThreads) {
    const int end = cu[i + 1];
    if (end <= t0) ++before;
    else if (end < t1) atomicAdd(cnt_s + (end - t0), 1);
  }
  before = __reduce_add_sync(0xffffffffu, before);
  if ((tid & 31) == 0 && before > 0) atomicAdd(cnt_s, before);
  __syncthreads();
  if (tid >= kWindow) return 0;
  int x = cnt_s[tid];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (tid >= o) x += y;
  }
  return x;
}

// Programmatic launch: this kernel may have started while the one before it
// ends.  Everything that it reads may still be written then, by a kernel of the
// library or of the caller: lengths, offsets and tables as well as the cache.  Here
// and in the attention kernels all of it is read with ordinary loads, after the
// wait: read-only ones (__ldg) are for data that nothing changes while the kernel
// runs, and may be moved before the wait.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel may start while this one runs (and waits in the same way).
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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

// Eight consecutive elements of a row as loaded.  amax: the larger of `a` and
// every |x| (NaN is passed over).
template <typename T>
struct Vec8;

template <>
struct Vec8<__nv_bfloat16> {
  using Max = __nv_bfloat162;
  uint4 w;
  __device__ __forceinline__ void load(const uint8_t* p) {
    w = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
  }
  __device__ __forceinline__ float2 pair(int i) const {
    const uint32_t u = word(i);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  static __device__ __forceinline__ Max none() { return __float2bfloat162_rn(0.f); }
  __device__ __forceinline__ Max amax(Max a) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = word(i);
      a = __hmax2(a, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u)));
    }
    return a;
  }
  static __device__ __forceinline__ float top(Max a) {
    return fmaxf(__low2float(a), __high2float(a));
  }
};

template <>
struct Vec8<float> {
  using Max = float;
  float4 a, b;
  __device__ __forceinline__ void load(const uint8_t* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ float2 pair(int i) const {
    return i == 0 ? make_float2(a.x, a.y) : i == 1 ? make_float2(a.z, a.w)
         : i == 2 ? make_float2(b.x, b.y) : make_float2(b.z, b.w);
  }
  static __device__ __forceinline__ Max none() { return 0.f; }
  __device__ __forceinline__ Max amax(Max m) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = pair(i);
      m = fmaxf(m, fmaxf(fabsf(x.x), fabsf(x.y)));
    }
    return m;
  }
  static __device__ __forceinline__ float top(Max m) { return m; }
};

// One warp's work on one unit: where it reads and writes, and its scale.
template <typename T>
struct Unit {
  const uint8_t* src;  // the run's first row of the head
  uint8_t* dst;        // row 0 of the block
  float* scale;
  float old;           // the block's scale (blocks with earlier tokens)
  int off, nv;         // rows before the run; vectors of the run

  // unit u of the window: runs, then K / V, then heads
  __device__ __forceinline__ void find(const WriteParams& p, const int4* run_s, int u, int vpr) {
    const int ri = u / (2 * p.n_kv);
    const int rem = u - ri * 2 * p.n_kv;
    const bool is_v = rem >= p.n_kv;
    const int h = is_v ? rem - p.n_kv : rem;
    const int4 run = run_s[ri];
    off = run.z;
    nv = run.y * vpr;
    scale = (is_v ? p.v_scales : p.k_scales) + int64_t(run.w) * p.n_kv + h;
    src = (is_v ? p.v : p.k) + (int64_t(run.x) * p.n_kv + h) * p.hd * sizeof(T);
    dst = (is_v ? p.v_pool : p.k_pool) + (int64_t(run.w) * p.bs * p.n_kv + h) * p.hd;
  }
  // the scale for magnitudes up to `a`
  __device__ __forceinline__ float fit(float a) const {
    // non-negative floats order as their bits
    a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
    const float f = fp8_scale_for(a);
    return off > 0 ? fmaxf(old, f) : f;
  }
  __device__ __forceinline__ void put(const Vec8<T>& v, int e, int vpr, int64_t dst_row,
                                      float inv) const {
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = v.pair(j);
      q[j] = e4m3x2(f.x * inv, f.y * inv);
    }
    const int r = e / vpr;
    *reinterpret_cast<uint2*>(dst + (off + r) * dst_row + (e - r * vpr) * 8) =
        make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
  }
  // the new scale; earlier rows move to it if it is larger
  __device__ __forceinline__ void finish(float s, float inv, int vpr, int64_t dst_row) const {
    const int lane = threadIdx.x & 31;
    if (off > 0 && s != old) {
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
};

// VPR: 8-element vectors of a head's row (0: read from p.hd).  MU: units that
// a warp takes at once, each with kHeld / MU vectors a lane (enough for 16
// rows of VPR vectors); larger units are read twice.
//
// A CTA column (x) finds the runs of its window of tokens; the warps of its
// grid.y CTAs share the units.  Four CTAs of 8 warps fit an SM (bf16), with
// 2-4 KB in flight per warp.
template <typename T, int VPR, int MU>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2)
    kv_write_fp8_kernel(const WriteParams p) {
  __shared__ int cnt_s[kWindow];
  __shared__ int4 run_s[kWindow];  // first token, tokens, offset in the block, block
  __shared__ int runs_s;
  pdl_wait();
  pdl_launch_dependents();
  const int t0 = blockIdx.x * kWindow;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = window_seq(p.cu, p.num_seqs, t0, cnt_s);
  if (warp == 0) {
    // a run: the new tokens of one sequence in one block.  Lane i looks at
    // token t0 + i: it begins a run if it is its sequence's first new token
    // or the first of a block.
    const int t = t0 + lane;
    int4 run = make_int4(0, 0, 0, 0);
    bool begins = false;
    if (t < p.num_tokens) {
      if (b >= p.num_seqs) {
        report(p.err, PKV_DEVERR_LENGTH);  // offsets that stop short of the token count
      } else {
        const int start = p.cu[b], end = p.cu[b + 1];
        const int L = p.seq_lens[b];
        const int64_t pos = int64_t(L) - end + t;
        if (start < 0 || t < start || t >= end || end > p.num_tokens || L < 0 || end - start > L) {
          report(p.err, PKV_DEVERR_LENGTH);
        } else if (pos / p.bs >= p.W) {
          report(p.err, PKV_DEVERR_TABLE_WIDTH);
        } else {
          const int off = static_cast<int>(pos % p.bs);
          begins = t == start || off == 0;
          if (begins) {
            const int blk = p.bt[int64_t(b) * p.W + pos / p.bs];
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
  } else if (threadIdx.x == 32 && blockIdx.x == 0 && blockIdx.y == 0) {
    if (p.cu[p.num_seqs] > p.num_tokens) report(p.err, PKV_DEVERR_LENGTH);
  }
  __syncthreads();

  constexpr int PU = kHeld / MU;  // vectors a lane holds of a unit
  const int vpr = VPR > 0 ? VPR : p.hd / 8;
  const int units = runs_s * 2 * p.n_kv;
  const int64_t src_row = int64_t(p.n_kv) * p.hd * sizeof(T);
  const int64_t dst_row = int64_t(p.n_kv) * p.hd;
  for (int u = (blockIdx.y * kWarps + warp) * MU; u < units; u += gridDim.y * kWarps * MU) {
    Unit<T> un[MU];
    Vec8<T> v[MU][PU];
    // (past the unit's end the last vector again, which changes no maximum: a
    // load behind a condition is waited for where it is issued)
    auto load = [&](int m, int base) {
#pragma unroll
      for (int i = 0; i < PU; ++i) {
        const int e = min(base + i * 32 + lane, un[m].nv - 1);
        const int r = e / vpr;
        v[m][i].load(un[m].src + r * src_row + (e - r * vpr) * 8 * sizeof(T));
      }
    };
#pragma unroll
    for (int m = 0; m < MU; ++m) {
      un[m].find(p, run_s, min(u + m, units - 1), vpr);
      un[m].old = *un[m].scale;
      load(m, 0);
    }
#pragma unroll
    for (int m = 0; m < MU; ++m) {
      if (u + m >= units) break;
      typename Vec8<T>::Max a = Vec8<T>::none();
      for (int base = 0;;) {
#pragma unroll
        for (int i = 0; i < PU; ++i) a = v[m][i].amax(a);
        if ((base += PU * 32) >= un[m].nv) break;
        load(m, base);
      }
      const float s = un[m].fit(Vec8<T>::top(a));
      const float inv = 1.f / s;  // exact: s is a power of two
      const bool again = un[m].nv > PU * 32;  // too large to hold
      for (int base = 0; base < un[m].nv; base += PU * 32) {
        if (again) load(m, base);
#pragma unroll
        for (int i = 0; i < PU; ++i) {
          const int e = base + i * 32 + lane;
          if (e < un[m].nv) un[m].put(v[m][i], e, vpr, dst_row, inv);
        }
      }
      un[m].finish(s, inv, vpr, dst_row);
    }
  }
}

// ------------------------------------------------------------------ gather

constexpr int kGatherRows = 4;   // rows a warp reads at once
constexpr int kGatherSteps = 2;  // and steps of 32 items in each

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

// An item: as many elements as fill one 16-byte store, so that a warp's stores
// are contiguous (16 elements an item would store them in strided pieces:
// 3.5 TB/s for fp32).
template <typename T>
struct Item;

template <>
struct Item<float> {
  using Load = uint32_t;  // 4 elements
  static __device__ __forceinline__ void store(uint8_t* dst, uint32_t u, float s) {
    const float2 a = e4m3x2_to_float2(static_cast<uint16_t>(u));
    const float2 b = e4m3x2_to_float2(static_cast<uint16_t>(u >> 16));
    __stcs(reinterpret_cast<float4*>(dst), make_float4(a.x * s, a.y * s, b.x * s, b.y * s));
  }
};

template <>
struct Item<__nv_bfloat16> {
  using Load = uint2;  // 8 elements (their values are bf16 numbers: nothing is rounded)
  static __device__ __forceinline__ void store(uint8_t* dst, uint2 u, float s) {
    const float2 a = e4m3x2_to_float2(static_cast<uint16_t>(u.x));
    const float2 b = e4m3x2_to_float2(static_cast<uint16_t>(u.x >> 16));
    const float2 c = e4m3x2_to_float2(static_cast<uint16_t>(u.y));
    const float2 d = e4m3x2_to_float2(static_cast<uint16_t>(u.y >> 16));
    __stcs(reinterpret_cast<uint4*>(dst),
           make_uint4(pack_bf16x2(a.x * s, a.y * s), pack_bf16x2(b.x * s, b.y * s),
                      pack_bf16x2(c.x * s, c.y * s), pack_bf16x2(d.x * s, d.y * s)));
  }
};

// A CTA reads back kWindow tokens: 2 x kWindow rows of n_kv x hd
// elements (K and V), kGatherRows rows of a warp at a time with
// kGatherRows x kGatherSteps loads in flight per lane.
template <typename T>
__global__ void __launch_bounds__(kThreads) kv_gather_fp8_kernel(const GatherParams p) {
  __shared__ int cnt_s[kWindow];
  __shared__ int blk_s[kWindow], off_s[kWindow];
  // The next kernel is not let in early: a planned decode of the bf16 cache reads
  // its first K/V before it waits, and these outputs may be that cache's blocks.
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
        const int pos = t0 + i - p.cu[b];
        if (pos < 0 || pos >= p.seq_lens[b]) {
          report(p.err, PKV_DEVERR_LENGTH);
        } else if (pos / p.bs >= p.W) {
          report(p.err, PKV_DEVERR_TABLE_WIDTH);
        } else {
          blk = p.bt[int64_t(b) * p.W + pos / p.bs];
          off = pos % p.bs;
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
  constexpr int E = sizeof(Load);  // elements per item, one byte each
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ipr = p.n_kv * p.hd / E;  // items of a row
  const int iph = p.hd / E;           // and of a head
  const bool pow2 = (iph & (iph - 1)) == 0;
  const int shift = 31 - __clz(iph);
  // rows 0 .. n - 1 are K's, n .. 2 n - 1 V's
  for (int r0 = warp * kGatherRows; r0 < 2 * n; r0 += kWarps * kGatherRows) {
    const uint8_t* src[kGatherRows];
    const float* scale[kGatherRows];
    uint8_t* dst[kGatherRows];
    bool have[kGatherRows];
#pragma unroll
    for (int k = 0; k < kGatherRows; ++k) {
      const int r = min(r0 + k, 2 * n - 1);  // past the last row: it again
      const bool is_v = r >= n;
      const int t = is_v ? r - n : r;
      have[k] = blk_s[t] >= 0;
      const int64_t blk = max(blk_s[t], 0);
      src[k] = (is_v ? p.v_pool : p.k_pool) + (blk * p.bs + off_s[t]) * ipr * E;
      scale[k] = (is_v ? p.v_scales : p.k_scales) + blk * p.n_kv;
      dst[k] = (is_v ? p.v_out : p.k_out) + int64_t(t0 + t) * ipr * 16;
    }
    for (int c0 = lane; c0 < ipr; c0 += 32 * kGatherSteps) {
      Load w[kGatherRows][kGatherSteps];
      float s[kGatherRows][kGatherSteps];
#pragma unroll
      for (int q = 0; q < kGatherSteps; ++q) {
        const int c = min(c0 + 32 * q, ipr - 1);
        const int h = pow2 ? c >> shift : c / iph;
#pragma unroll
        for (int k = 0; k < kGatherRows; ++k) {
          w[k][q] = __ldcs(reinterpret_cast<const Load*>(src[k]) + c);
          s[k][q] = scale[k][h];
        }
      }
#pragma unroll
      for (int q = 0; q < kGatherSteps; ++q) {
        const int c = c0 + 32 * q;
        if (c < ipr) {
#pragma unroll
          for (int k = 0; k < kGatherRows; ++k)
            if (r0 + k < 2 * n) Item<T>::store(dst[k] + int64_t(c) * 16, have[k] ? w[k][q] : Load{}, have[k] ? s[k][q] : 0.f);
        }
      }
    }
  }
}

// Self-test of the 8-bit kernels' waits: a warp half of whose lanes wait for a
// phase that is complete and half for one that nothing completes, for at most
// `polls` polls.  The lanes that give up report the timeout (err) and tell the
// CTA; err is left clear if some lane is told otherwise than its warp.
__global__ void fp8_wait_selftest_kernel(uint32_t polls, int32_t* err) {
  __shared__ uint64_t bars[2];
  __shared__ int flag, reported;
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
    mbar_init(bars, 1);
    mbar_init(bars + 1, 1);
    flag = reported = 0;
    fence_barrier_init();
    mbar_arrive(bars);
  }
  __syncwarp();
  const bool there = warp_wait_or_abort(bars, 0, &flag, polls);
  const bool mixed = warp_wait_or_abort(bars + (lane & 1), 0, &flag, polls);
  const bool quiet = flag == 0;
  __syncwarp();
  wait_or_flag(bars + (lane & 1), 0, &flag, &reported, polls);
  __syncwarp();
  // (the flag is set: this ends at once, not after the kernels' own limit)
  const bool told = warp_wait_or_abort(bars + (lane & 1), 0, &flag);
  if (__all_sync(0xffffffffu, there && !mixed && quiet && flag == 1 && !told) && lane == 0)
    report(err, reported);
}

}  // namespace

cudaError_t launch_fp8_bounded_wait_selftest(uint32_t polls, int32_t* err, cudaStream_t stream) {
  fp8_wait_selftest_kernel<<<1, 32, 0, stream>>>(polls, err);
  return cudaGetLastError();
}

template <typename T>
static cudaError_t write_as(const WriteParams& p, dim3 grid, cudaStream_t stream) {
  // two units at once where 16 rows of a head are at most half of what a warp
  // holds, and blocks have no more rows than that
  auto kern = kv_write_fp8_kernel<T, 0, 1>;
  if (p.bs <= 16 && p.hd == 16) kern = kv_write_fp8_kernel<T, 2, 2>;
  else if (p.bs <= 16 && p.hd == 32) kern = kv_write_fp8_kernel<T, 4, 2>;
  else if (p.bs <= 16 && p.hd == 64) kern = kv_write_fp8_kernel<T, 8, 2>;
  else if (p.hd == 128) kern = kv_write_fp8_kernel<T, 16, 1>;
  return launch_pdl(kern, grid, kThreads, 0, stream, p);
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
  // A window holds about kWindow / block_size + 1 + kWindow * num_seqs /
  // num_tokens runs.  Few windows (a decode step): CTAs enough that each warp
  // has about one unit.  Many (prompts): one CTA a window, so that what it
  // takes to find the runs is paid once for all their units (31,722 tokens of
  // 8 x 64: 63 us with four CTAs for each window of 16).
  const int64_t windows = (int64_t(num_tokens) + kWindow - 1) / kWindow;
  const int64_t runs = std::min<int64_t>(
      std::min(kWindow, num_tokens),
      kWindow / pool.block_size + 1 + int64_t(kWindow) * num_seqs / num_tokens);
  const int64_t most = (runs * 2 * pool.n_kv + kWarps - 1) / kWarps;
  const int64_t want = (int64_t(sm_count()) * 4 + windows - 1) / windows;
  const dim3 grid(static_cast<unsigned>(windows),
                  static_cast<unsigned>(std::min<int64_t>(std::min(most, want), 1024)));
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
  const unsigned grid = static_cast<unsigned>((int64_t(total_tokens) + kWindow - 1) /
                                              kWindow);
  return launch_pdl(dtype == PKV_F32 ? kv_gather_fp8_kernel<float>
                                     : kv_gather_fp8_kernel<__nv_bfloat16>,
                    dim3(grid), kThreads, 0, stream, p);
}

}  // namespace pkv
