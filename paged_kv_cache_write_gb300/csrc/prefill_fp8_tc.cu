// Chunked prefill over the 8-bit cache on the 5th-generation tensor cores:
// bf16 queries, head_dim 64 / 128.
//
// What is computed: query i of a chunk of c queries at the end of an L-token
// sequence attends keys 0 .. L - c + i of its KV head, with element = e4m3
// value x scale of (block, head).  With the byte values k8, v8 of a block:
//   x = (q . k8) * (scale * log2 e * ks),  w = 2^(x + log2 vs - M + 4),
//   l += (sum of the block's w) / vs,  O += w v8,  out = O / l.
// M is a running reference of x + log2 vs, moved to the maximum when a weight
// would pass f16's 65,504 (the maximum has grown 2^12-fold: seldom after
// the first tile; f16 is normal down to 2^-18 of the reference's weight).  Scales cost
// nothing per element: they are constants of a 16-key block.
//
// tcgen05 takes no f16 x e4m3 product, so the cache's bytes become f16 (exact)
// on their way into shared memory.  Queries become f16 too, each row times
// the power of two that brings its largest element to 2^14 .. 2^15 (exact for
// bf16 within 2^28 of it; undone in the score's factor).
//
// One CTA per SM owns two 128-row tiles, A and B, of one (sequence, KV head);
// a row is one (query, query head) pair.  Keys go in tiles of 64 (4 blocks), so
// that scores have two buffers per row tile in TMEM: while a tile's softmax
// runs, its next scores are computed, and neither waits for the other.
//  warps 0-3    softmax of tile A, 4-7 of tile B: one thread per row.  Weights
//               are computed against the reference as it stands; only if some
//               weight came out past f16's range (their partial sums tell) the
//               maximum is taken, the reference moved to it and the tile done
//               again, so that most tiles need no maximum at all.  Weights go
//               back to TMEM as f16 over the scores.
//  warps 8, 9   issue the MMAs of tiles A and B, one elected lane each: S_X of
//               the first two key tiles, then for each key tile j, once its
//               weights are there, O_X += W_X V_j and S_X = Q_X K_{j+2}^T.
//               (A look at a barrier takes the issuing lane 120 cycles, a step's
//               MMAs 600: one lane for both tiles left the tensor core idle
//               half of the time.)  Warp 8 allocates TMEM: 2 S_A, 2 S_B, O_A,
//               O_B, all 512 columns at head_dim 128.
//  warps 10-15  bring K and V, a block (16 tokens) at a time in turn: 16-byte
//               loads straight from the pool, each warp's next two blocks on
//               their way, e4m3 -> f16 in registers, 128-byte-swizzled tiles
//               in four-stage rings.
// Two row tiles a CTA, because they share the conversion of K and V: CTAs of one
// row tile, two on an SM, took 381 us for 214 (32 heads on 8, 4 chunks of 512
// after 2,048 - 8,192 tokens of head_dim 128).
//
// Measured: 4 chunks of 512 after 990 - 3,018 tokens, 64 heads of 128 on 8,
// 159 us (936 TFLOP/s); 2 chunks of 2,048 ending at 8,192, 823 us (1,168);
// head_dim 64, 32 heads on 8, 4 chunks of 1,024 ending at 4,096, 226 us (533).
// Bound by the softmax warps, some 1,800 cycles a key tile of 64 (MMAs: 1,330 at
// head_dim 128), and by 10,000 cycles of each CTA that are not its loop: work
// order 2,500, set-up 500, queries 3,000 - 6,000, first scores 1,500, output
// 2,000 - 4,000.
//
// 16 warps leave 128 registers a thread, and no loop may spill: with 200 KB of
// shared memory little L1 is left, and a reload from local memory costs an L2
// round trip.
//
// Values past the sequence's end are stored as zeros.  A NaN value that some
// row of the tile may not see is stored as zero too, and its dim and first
// position noted: rows that do see it get NaN at the end.  Every wait is
// bounded; a thread that gave up still takes part in the CTA's barriers.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "device.cuh"
#include "fp8.cuh"
#include "host_cache.h"
#include "launch.h"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kRows = 128;
constexpr int kTileKeys = 64;
constexpr int kBlk = 16;
constexpr int kBlocks = kTileKeys / kBlk;  // blocks per key tile
static_assert(kBlocks == 4, "units and score chunks below");
constexpr int kMmaWarp = 8;  // and 9, after eight of the softmax
constexpr int kLoadWarp0 = 10;
constexpr int kLoadWarps = 6;
constexpr int kAhead = 2;  // blocks in flight per load warp
constexpr int kThreads = 16 * 32;
constexpr int kStages = 4;
constexpr int kScaleStages = 8;  // scales outlive their K stage (see the load warps)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kWeightLog2 = 4.f;     // log2 of the reference's weight
constexpr float kWeightMax = 65504.f;  // f16's largest
constexpr uint32_t kTmemCols = 512;

struct TcParams {
  const __nv_bfloat16* q;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const float* k_scales;
  const float* v_scales;
  const int32_t* bt;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  __nv_bfloat16* out;
  int32_t* err;
  int B, n_heads, n_kv, rep, rep_inv, W, num_blocks, max_len, total_q, q_per_tile;
  int ordered, last_seq;
  ChunkLimits limits;
  float scale_log2;
};

template <int HD>
struct Layout {
  static constexpr int NH = HD / 64;               // 128-byte column halves
  static constexpr int Q_HALF = kRows * 128;       // 16 KB
  static constexpr int KV_HALF = kTileKeys * 128;  // 8 KB
  static constexpr int Q_TILE = NH * Q_HALF;
  static constexpr int KV_TILE = NH * KV_HALF;
  static constexpr int K_OFF = 2 * Q_TILE;  // after Q_A, Q_B
  static constexpr int V_OFF = K_OFF + kStages * KV_TILE;
  static constexpr int SCALE_OFF = V_OFF + kStages * KV_TILE;  // ks, lv, 1/vs [stages][4]
  static constexpr int NAN_OFF = SCALE_OFF + 3 * kScaleStages * kBlocks * 4;  // [HD] + flag
  static constexpr int BAR_OFF = (NAN_OFF + HD * 4 + 16 + 15) / 16 * 16;
  static constexpr int BYTES = BAR_OFF + 512;
  // + 1 KB alignment slack; at least 120 KB so only one CTA fits per SM (it
  // takes all 512 TMEM columns)
  static constexpr int REQUEST = (BYTES + 1024) > 120 * 1024 ? (BYTES + 1024) : 120 * 1024;
};

// Instruction descriptor of kind::f16 with f16 A and B (format bits 0), fp32
// accumulator; b_mn: B stored MN-major.
constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn) {
  return (1u << 4) | (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}


// Whether the barrier's phase of this parity is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_fp8_tc_kernel(const TcParams p) {
  using Lay = Layout<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);

  asm volatile("griddepcontrol.wait;" ::: "memory");  // the preceding kernel's results
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Work order, as in the bf16 prefill: with at most blockDim.x sequences, x
  // numbers the (sequence, KV head, tile pair) triples, sequences by
  // descending work and each one's pairs from the last (most keys) down;
  // otherwise z, y, x in the natural order.  Work values are staged in the
  // (still unused) V stages.
  __shared__ int order_s, pair_s, head_s, seq_s[3], job_s[4];  // seq_s: cu_q of both ends, length
  int g = blockIdx.y;
  int b = blockIdx.z, pair = blockIdx.x;
  if (p.ordered) {
    const int t = threadIdx.x;
    int64_t* work_s = reinterpret_cast<int64_t*>(smem + Lay::V_OFF);
    int* pairs_s = reinterpret_cast<int*>(work_s + p.B);
    const int qpp = 2 * p.q_per_tile;
    int64_t wt = 0;
    int pt = 0, at = 0, end = 0, len = 0;
    if (t < p.B) {
      at = p.cu_q[t];
      end = p.cu_q[t + 1];
      len = p.seq_lens[t];
      if (blockIdx.x == 0) report_bad_chunk(p.err, p.limits, at, end, len, t == p.last_seq);
      const int64_t cs = int64_t(end) - at;
      const int64_t Ls = min(len, p.max_len);
      wt = cs * (2 * Ls - cs + 1);
      pt = cs > 0 ? static_cast<int>((cs + qpp - 1) / qpp) : 0;
      work_s[t] = wt;
      pairs_s[t] = pt;
    }
    if (t == 0) order_s = -1;
    __syncthreads();
    if (t < p.B) {  // the sequence's first slot: the (head, pair) slots of the heavier ones
      int64_t first = 0;
#pragma unroll 8
      for (int s = 0; s < p.B; ++s) {
        const int64_t ws = work_s[s];
        if (ws > wt || (ws == wt && s < t)) first += pairs_s[s];
      }
      const int64_t x = blockIdx.x;
      const int64_t lo = first * p.n_kv, n = int64_t(pt) * p.n_kv;
      if (x >= lo && x < lo + n) {
        const int off = static_cast<int>(x - lo);
        order_s = t;
        seq_s[0] = at;
        seq_s[1] = end;
        seq_s[2] = len;
        head_s = off / pt;
        pair_s = pt - 1 - (off - (off / pt) * pt);
      }
    }
    __syncthreads();
    if (order_s < 0) return;  // slot past the last pair
    b = order_s;
    g = head_s;
    pair = pair_s;
  } else {
    if (threadIdx.x == 0) {
      seq_s[0] = p.cu_q[b];
      seq_s[1] = p.cu_q[b + 1];
      seq_s[2] = p.seq_lens[b];
      if (pair == 0 && g == 0)
        report_bad_chunk(p.err, p.limits, seq_s[0], seq_s[1], seq_s[2], b == p.last_seq);
    }
    __syncthreads();
  }
  const int q0 = seq_s[0];
  // idle CTAs leave before any barrier or TMEM use
  if (q0 < 0 || seq_s[1] <= q0 || seq_s[1] > p.total_q) return;  // no chunk, or not within the rows
  const int c = seq_s[1] - q0;
  const int i0 = pair * 2 * p.q_per_tile;  // first query of tile A
  if (i0 >= c) return;
  const int L = min(seq_s[2], p.max_len);
  if (L < c) return;
  const int i_end = min(c, i0 + 2 * p.q_per_tile);
  const int n_tiles = (L - c + i_end - 1) / kTileKeys + 1;
  const int n_blocks_seq = (L + kBlk - 1) / kBlk;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::BAR_OFF);
  uint64_t* q_full = bars + 0;         // [2] per row tile
  uint64_t* k_full = bars + 2;         // [4] per stage
  uint64_t* k_empty = bars + 6;        // [4]
  uint64_t* v_full = bars + 10;        // [4]
  uint64_t* v_empty = bars + 14;       // [4]
  uint64_t* s_full = bars + 18;        // [row tile][buffer]
  uint64_t* w_ready = bars + 22;       // [row tile][buffer]
  uint64_t* o_done = bars + 26;        // [row tile][key tile % 2], the last two tiles
  uint64_t* drain = bars + 30;         // [2] per row tile
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 32);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* ks_s = reinterpret_cast<float*>(smem + Lay::SCALE_OFF);  // [kScaleStages][4]
  float* lv_s = ks_s + kScaleStages * kBlocks;
  float* iv_s = lv_s + kScaleStages * kBlocks;
  int* nan_s = reinterpret_cast<int*>(smem + Lay::NAN_OFF);    // [HD] first NaN position
  int* nan_any = nan_s + HD;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // every wait is one of these two: bounded, by a whole warp or by one lane
  auto wait_one = [&](uint64_t* bar, uint32_t parity) {
    return wait_or_abort(bar, parity, abort_flag);
  };
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    return warp_wait_or_abort(bar, parity, abort_flag);
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(q_full + i, 4);
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(w_ready + i, 4);
      mbar_init(o_done + i, 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(k_full + i, kBlocks);
      mbar_init(k_empty + i, 2);  // left by both row tiles
      mbar_init(v_full + i, kBlocks);
      mbar_init(v_empty + i, 2);
    }
    mbar_init(drain, 1);
    mbar_init(drain + 1, 1);
    *abort_flag = 0;
    *nan_any = 0;
    job_s[0] = i0;
    job_s[1] = c;
    job_s[2] = q0;
    job_s[3] = g;
    fence_barrier_init();
  }
  if (threadIdx.x < HD) nan_s[threadIdx.x] = INT_MAX;
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  auto q_tile = [&](int x) { return smem + x * Lay::Q_TILE; };
  auto k_st = [&](int j) { return smem + Lay::K_OFF + (j % kStages) * Lay::KV_TILE; };
  auto v_st = [&](int j) { return smem + Lay::V_OFF + (j % kStages) * Lay::KV_TILE; };
  auto s_tm = [&](int x, int j) { return tmem + uint32_t(x * 2 + (j & 1)) * kTileKeys; };
  auto o_tm = [&](int x) { return tmem + 256u + uint32_t(x) * 128u; };

  if (warp >= kLoadWarp0) {
    // ------------------------------------------------------ K and V tiles
    // Unit 8 j + i is block i of K tile j, unit 8 j + 4 + i of V tile j; the
    // warps take them in turn.  A step of the warp covers 32 / PR rows; lane:
    // 16-byte piece lane % PR.  At head_dim 128 the lanes of a row's second
    // half take their piece from the row's neighbour, so that the eight lanes
    // of a store phase, whose pieces are then even ones of one row and odd ones
    // of the other, touch each bank once.
    constexpr int PR = HD / 16;    // pieces of a row
    constexpr int RS = 32 / PR;    // rows per step: 4 or 8
    constexpr int NV = kBlk / RS;  // steps: 4 or 2
    const int piece = lane % PR, half = piece >> 2;
    const int r0 = HD == 128 ? (lane / PR) ^ half : lane / PR;  // row of step 0
    const int32_t* row = p.bt + int64_t(b) * p.W;
    const int pitch = p.n_kv * HD;
    const int lane_off = r0 * pitch + g * HD + piece * 16;
    const int step_off = RS * pitch;
    // where the lane's piece (16 dims: two 16-byte pieces of f16) goes in row
    // r0 + RS i of a block: (r0 + RS i) % 8 is r0, and r0 + 4 in odd steps of 4
    const int at = (piece & 3) * 2;
    const int put_lo = half * Lay::KV_HALF + r0 * 128 + ((at ^ r0) << 4);
    const int put_hi = half * Lay::KV_HALF + r0 * 128 + (((at + 1) ^ r0) << 4);
    const int n_units = 2 * kBlocks * n_tiles;
    // -1: the sequence has no block there
    auto id_of = [&](int u) {
      const int jb = (u >> 3) * kBlocks + (u & 3);
      int id = -1;
      if (u < n_units && jb < n_blocks_seq) id = row[jb];
      return id;
    };
    uint4 d[kAhead][NV];
    float sk[kAhead], sv[kAhead];  // scales of a K unit's block (every lane alike)
    int id_d[kAhead], id_next[kAhead];
    // (unconditional loads, of block 0 where there is none, so that they stay
    // in flight: a selected load is waited for where it is issued)
    auto fetch = [&](uint4 (&x)[NV], float& ks, float& vs, int& id, int u) {
      if (id >= p.num_blocks || id < 0) id = -1;
      const int blk = max(id, 0);
      const uint8_t* src = ((u & 4) ? p.v_pool : p.k_pool) + int64_t(blk) * (kBlk * pitch) + lane_off;
#pragma unroll
      for (int i = 0; i < NV; ++i) x[i] = *reinterpret_cast<const uint4*>(src + i * step_off);
      if (!(u & 4)) {
        ks = p.k_scales[int64_t(blk) * p.n_kv + g];
        vs = p.v_scales[int64_t(blk) * p.n_kv + g];
      }
    };
    const int w = warp - kLoadWarp0;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int u = w + k * kLoadWarps;
      id_d[k] = id_of(u);
      fetch(d[k], sk[k], sv[k], id_d[k], u);
      id_next[k] = id_of(u + kAhead * kLoadWarps);
    }
    bool ok = true;
    for (int u0 = w; u0 < n_units && ok; u0 += kAhead * kLoadWarps) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int u = u0 + k * kLoadWarps;
        if (u >= n_units || !ok) break;
        const int j = u >> 3, bi = u & 3;
        const bool is_v = (u & 4) != 0;
        const int st = j % kStages;
        const uint32_t use = j / kStages;
        if (use > 0 && !wait_all((is_v ? v_empty : k_empty) + st, (use - 1) & 1)) {
          if (lane == 0) {
            report(p.err, PKV_DEVERR_TIMEOUT);
            *abort_flag = 1;
          }
          ok = false;
          break;
        }
        const int pos0 = (j * kBlocks + bi) * kBlk;
        if (!is_v && lane == 0) {
          // The scales of tile j - 8 are no longer read: K stage j was free, so
          // S_{j-4} is complete, which was issued once W_{j-6} was there.
          const int o = (j % kScaleStages) * kBlocks + bi;
          const bool good = id_d[k] >= 0;
          if (!good && pos0 < L) report(p.err, PKV_DEVERR_BLOCK_ID);  // (a block that it holds)
          ks_s[o] = good ? sk[k] : 1.f;
          lv_s[o] = good ? __log2f(sv[k]) : 0.f;
          iv_s[o] = good ? __fdividef(1.f, sv[k]) : 1.f;
        }
        if (id_d[k] < 0 || pos0 + kBlk > L) {
          // what lies past the sequence's end, and a bad block, is zeros
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (id_d[k] < 0 || pos0 + r0 + RS * i >= L) d[k][i] = make_uint4(0u, 0u, 0u, 0u);
        }
        if (is_v && pos0 + kBlk > L - c + i0 + 1) {
          // some row may not see some key of this block: take out its NaNs
          const int first_last = L - c + i0;  // the last key that the pair's first query sees
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int pos = pos0 + r0 + RS * i;
            uint32_t v4[4] = {d[k][i].x, d[k][i].y, d[k][i].z, d[k][i].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t bad = __vcmpeq4(v4[q] & 0x7f7f7f7fu, 0x7f7f7f7fu);
              if (bad != 0 && pos > first_last) {
                for (int e = 0; e < 4; ++e)
                  if ((bad >> (8 * e)) & 1u) atomicMin(nan_s + piece * 16 + 4 * q + e, pos);
                v4[q] &= ~bad;
                atomicOr(nan_any, 1);
              }
            }
            d[k][i] = make_uint4(v4[0], v4[1], v4[2], v4[3]);
          }
        }
        uint8_t* base = (is_v ? v_st(j) : k_st(j)) + bi * (kBlk * 128);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const uint32_t x[4] = {d[k][i].x, d[k][i].y, d[k][i].z, d[k][i].w};
          uint32_t f[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            f[2 * q] = e4m3x2_to_f16x2(static_cast<uint16_t>(x[q]));
            f[2 * q + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(x[q] >> 16));
          }
          // piece q of row r sits at q ^ (r % 8)
          const int odd4 = (RS * i) & 4 ? 64 : 0;
          uint8_t* dst = base + i * RS * 128;
          *reinterpret_cast<uint4*>(dst + (put_lo ^ odd4)) = make_uint4(f[0], f[1], f[2], f[3]);
          *reinterpret_cast<uint4*>(dst + (put_hi ^ odd4)) = make_uint4(f[4], f[5], f[6], f[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive((is_v ? v_full : k_full) + st);
        const int un = u + kAhead * kLoadWarps;
        id_d[k] = id_next[k];
        fetch(d[k], sk[k], sv[k], id_d[k], un);
        id_next[k] = id_of(un + kAhead * kLoadWarps);
      }
    }
  } else if (warp >= kMmaWarp) {
    // ----------------------------------------------------------------- MMA
    // One elected lane.  (elect.sync, not a test of the lane: the compiler then
    // keeps descriptors in uniform registers, and an MMA takes some 30 cycles
    // to issue instead of 45.)
    if (elect_one()) {
      constexpr uint32_t idesc_qk = idesc_f16_f32(kRows, kTileKeys, false);
      constexpr uint32_t idesc_pv = idesc_f16_f32(kRows, HD, true);
      // descriptors of the tiles' starts; a step within a tile adds its byte
      // offset / 16 to the address field, which does not overflow
      const uint64_t q_desc = tc::sw128_desc(smem_addr(q_tile(0)), 16, 1024);
      const uint64_t k_desc = tc::sw128_desc(smem_addr(k_st(0)), 16, 1024);
      const uint64_t v_desc = tc::sw128_desc(smem_addr(v_st(0)), Lay::KV_HALF, 1024);
      auto issue_qk = [&](int x, int j) {
        const uint64_t qd = q_desc + uint32_t(x * Lay::Q_TILE) / 16;
        const uint64_t kd = k_desc + uint32_t((j % kStages) * Lay::KV_TILE) / 16;
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          tc::mma_ss(s_tm(x, j), qd + ((kk >> 2) * Lay::Q_HALF + (kk & 3) * 32) / 16,
                     kd + ((kk >> 2) * Lay::KV_HALF + (kk & 3) * 32) / 16, idesc_qk, kk > 0);
        tc::commit(s_full + x * 2 + (j & 1));
      };
      auto issue_pv = [&](int x, int j) {
        const uint64_t vd = v_desc + uint32_t((j % kStages) * Lay::KV_TILE) / 16;
#pragma unroll
        for (int kk = 0; kk < kTileKeys / 16; ++kk)
          // W: 16 f16 are 8 columns
          tc::mma_ts(o_tm(x), s_tm(x, j) + kk * 8, vd + kk * 2048 / 16, idesc_pv, j > 0 || kk > 0);
        if (j + 2 >= n_tiles) tc::commit(o_done + x * 2 + (j & 1));  // (see the softmax)
      };
      const int x = warp - kMmaWarp;
      bool ok = wait_one(q_full + x, 0);
      for (int j = 0; j < 2 && j < n_tiles && ok; ++j) {
        if (!(ok = wait_one(k_full + j, 0))) break;
        tc::fence_after_sync();
        issue_qk(x, j);
        tc::commit(k_empty + j);  // this row tile has read K_j
      }
      for (int j = 0; j < n_tiles && ok; ++j) {
        const int st = j % kStages, kn = (j + 2) % kStages;
        const bool more = j + 2 < n_tiles;
        // (the weights last: once they are there both products go at once)
        ok = wait_one(v_full + st, (j / kStages) & 1) &&
             (!more || wait_one(k_full + kn, ((j + 2) / kStages) & 1)) &&
             wait_one(w_ready + x * 2 + (j & 1), (j >> 1) & 1);
        if (!ok) break;
        tc::fence_after_sync();
        issue_pv(x, j);
        tc::commit(v_empty + st);
        if (!more) continue;
        issue_qk(x, j + 2);
        tc::commit(k_empty + kn);
      }
      if (!ok) {
        report(p.err, PKV_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      // every MMA issued above has finished before TMEM is released
      tc::commit(drain + x);
      for (uint32_t i = 0; i < kFp8Polls && !mbar_park(drain + x, 0); ++i) {
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax
    const int x = warp >> 2;               // tile A or B
    // (TMEM lane = row of the tile: (warp % 4) * 32 + lane)
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    // A row's 16-byte vectors of q (and of out) are RL = HD / 8 lanes' work: the
    // warp goes through its rows 32 / RL at a time, so that memory is touched
    // row by row (with every lane at a row of its own, 32 lines a load, one tile
    // of 64 tokens took 3 us longer).  Row `m` of the warp: its query,
    // or -1, and its first element; read from shared memory where it is needed,
    // so that it takes no registers in between.
    constexpr int RL = HD / 8, RG = 32 / RL, STEPS = 32 / RG;
    struct Row {
      int qi;
      int64_t off;
    };
    auto row_of = [&](int m) {
      const int* job = job_s;
      const int rr = (warp & 3) * 32 + m;
      const int q = (rr * p.rep_inv) >> 16;  // rr / p.rep
      const int qi = job[0] + x * p.q_per_tile + q;
      const bool active = q < p.q_per_tile && qi < job[1];
      return Row{active ? qi : -1,
                 (int64_t(job[2] + qi) * p.n_heads + job[3] * p.rep + (rr - q * p.rep)) * HD};
    };
    // where vector k of row m of the warp lies in the Q tile
    auto q_at = [&](int m, int k) {
      const int rr = (warp & 3) * 32 + m;
      return q_tile(x) + (k >> 3) * Lay::Q_HALF + rr * 128 + (((k & 7) ^ (rr & 7)) << 4);
    };
    int last, cut;   // last key that the row sees; the least of the warp's rows
    float rs = 1.f;  // undoes the row's power of two; times scale * log2 e
    {
      const Row me = row_of(lane);
      last = me.qi >= 0 ? L - c + me.qi : INT_MAX;  // a row without a query is never masked
      cut = __reduce_min_sync(0xffffffffu, last);
#pragma unroll
      for (int s0 = 0; s0 < STEPS; s0 += 8) {
        uint4 u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const Row o = row_of((s0 + i) * RG + lane / RL);
          u[i] = reinterpret_cast<const uint4*>(p.q + (o.qi >= 0 ? o.off : 0))[lane % RL];
          if (o.qi < 0) u[i] = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t e[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
          float a = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            a = fmaxf(a, fmaxf(fabsf(__uint_as_float(e[k] << 16)),
                               fabsf(__uint_as_float(e[k] & 0xffff0000u))));
#pragma unroll
          for (int o = 1; o < RL; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
          const int up = min(126, 14 + 127 - static_cast<int>(__float_as_uint(a) >> 23));
          const float f = pow2f(up);
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            o[k] = pack_f16x2(__uint_as_float(e[k] << 16) * f,
                              __uint_as_float(e[k] & 0xffff0000u) * f);
          *reinterpret_cast<uint4*>(q_at((s0 + i) * RG + lane / RL, lane % RL)) =
              make_uint4(o[0], o[1], o[2], o[3]);
          // the factor goes to the lane whose row it is
          const float back = __shfl_sync(0xffffffffu, pow2f(-up), (lane % RG) * RL);
          if (lane / RG == s0 + i) rs = back * p.scale_log2;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full + x);
    }
    float m_used = -INFINITY, l_sum = 0.f;
    bool ok = true;
    auto gave_up = [&]() {
      if (lane == 0) {
        report(p.err, PKV_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      ok = false;
    };
    uint32_t v[kTileKeys];  // scores
    auto request = [&](int j) {  // (there after tmem_wait_ld)
      tc::fence_after_sync();
      tc::tmem_ld32(s_tm(x, j) + lane_base, *reinterpret_cast<uint32_t(*)[32]>(v));
      tc::tmem_ld32(s_tm(x, j) + lane_base + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
    };
    auto s_bar = [&](int j) { return s_full + x * 2 + (j & 1); };
    if (wait_all(s_bar(0), 0)) request(0);
    else gave_up();
    for (int j = 0; j < n_tiles && ok; ++j) {
      const uint32_t s_addr = s_tm(x, j) + lane_base;
      const float* sc = ks_s + (j % kScaleStages) * kBlocks;
      const float4 k4 = *reinterpret_cast<const float4*>(sc);
      const float4 l4 = *reinterpret_cast<const float4*>(sc + kScaleStages * kBlocks);
      const float4 i4 = *reinterpret_cast<const float4*>(sc + 2 * kScaleStages * kBlocks);
      // (factors are > 0; none is zero: -inf stays -inf)
      const float factor[4] = {fmaxf(rs * k4.x, 1.2e-38f), fmaxf(rs * k4.y, 1.2e-38f),
                               fmaxf(rs * k4.z, 1.2e-38f), fmaxf(rs * k4.w, 1.2e-38f)};
      const float shift[4] = {l4.x, l4.y, l4.z, l4.w}, inv_vs[4] = {i4.x, i4.y, i4.z, i4.w};
      // A weight w is flushed 2^126 below 1, and counts in the sum as w / vs: beside
      // a value scale 2^80 times its own (up to 2^60) a key's share could be lost.
      // Tiles with such a scale take their sums from the scores, without scales.
      const bool far = fminf(fminf(l4.x, l4.y), fminf(l4.z, l4.w)) < -20.f;
      const int pos0 = j * kTileKeys;
      tc::tmem_wait_ld();
      if (pos0 + kTileKeys - 1 > cut) {  // keys past some row's causal limit
#pragma unroll
        for (int k = 0; k < kTileKeys; ++k)
          if (pos0 + k > last) v[k] = __float_as_uint(-INFINITY);
      }
      float d = 0.f, add = 0.f;  // d: log2 of the factor on what came before
      bool move = j == 0;     // set the reference to the maximum
      bool rescale = false;   // some row of the warp moved its reference
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
        if (move) {
          float mx = -INFINITY;  // of x + log2 vs
#pragma unroll
          for (int bk = 0; bk < kBlocks; ++bk) {
            float mb = __uint_as_float(v[bk * 16]);
#pragma unroll
            for (int k = 1; k < 16; ++k) mb = fmaxf(mb, __uint_as_float(v[bk * 16 + k]));
            mx = fmaxf(mx, fmaf(mb, factor[bk], shift[bk]));
          }
          const float m_new = fmaxf(m_used, mx);
          if (m_new > m_used) d = m_used - m_new;
          m_used = m_new;
        }
        rescale = pass > 0;
        const float mref = (m_used == -INFINITY ? 0.f : m_used) - kWeightLog2;
        float most = 0.f;
        add = 0.f;
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t pk[16];
#pragma unroll
          for (int bb = 0; bb < 2; ++bb) {
            const int bk = ch * 2 + bb;
            const float f = factor[bk], cst = shift[bk] - mref;
            const float2 f2 = make_float2(f, f), c2 = make_float2(cst, cst);
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int e = bk * 16 + 2 * k;
              const float2 t2 =
                  __ffma2_rn(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), f2, c2);
              const float2 pe = make_float2(fast_exp2(t2.x), fast_exp2(t2.y));
              acc = __fadd2_rn(acc, pe);
              pk[bb * 8 + k] = pack_f16x2(pe.x, pe.y);
            }
            add = fmaf(acc.x + acc.y, inv_vs[bk], add);
            most = fmaxf(most, fmaxf(acc.x, acc.y));  // no weight is larger
          }
          tc::tmem_st16(s_addr + ch * 16, pk);
        }
        if (far) {
          add = 0.f;
#pragma unroll
          for (int k = 0; k < kTileKeys; ++k)
            add += fast_exp2(fmaf(__uint_as_float(v[k]), factor[k / 16], -mref));
        }
        move = most > kWeightMax;
        if (!__any_sync(0xffffffffu, move)) break;
        tc::tmem_wait_st();  // the second pass stores to the same columns
      }
      // (2^d in two steps: it underflows where a value scale is some 2^100 times the
      // earlier ones, whose keys' share of the sum then still counts)
      l_sum = l_sum * fast_exp2(fminf(d + 100.f, 0.f)) * fast_exp2(fmaxf(d, -100.f)) + add;
      if (rescale && j > 0) {
        // O_X has to hold all products before this tile's.  S_{j+1} was computed
        // after them; only the last tiles have a barrier for it of their own.
        // (W_j is not there yet, so no later phase can have completed.)
        const bool there = j + 1 < n_tiles ? wait_all(s_bar(j + 1), ((j + 1) >> 1) & 1)
                                           : wait_all(o_done + x * 2 + ((j - 1) & 1), 0);
        if (!there) {
          gave_up();
          break;
        }
        tc::fence_after_sync();
        const float alpha = fast_exp2(d);
        const float2 a2 = make_float2(alpha, alpha);
#pragma unroll 1
        for (int ch = 0; ch < HD / 32; ++ch) {
          const uint32_t o_addr = o_tm(x) + lane_base + ch * 32;
          uint32_t ov[32];
          tc::tmem_ld32(o_addr, ov);
          tc::tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 o2 = __fmul2_rn(
                make_float2(__uint_as_float(ov[2 * k]), __uint_as_float(ov[2 * k + 1])), a2);
            ov[2 * k] = __float_as_uint(o2.x);
            ov[2 * k + 1] = __float_as_uint(o2.y);
          }
          tc::tmem_st32(o_addr, ov);
        }
      }
      // The next scores are mostly there (their product was issued a tile ago):
      // their load then overlaps the weights' store.
      const bool more = j + 1 < n_tiles;
      const bool early =
          more && __all_sync(0xffffffffu, mbar_test(s_bar(j + 1), ((j + 1) >> 1) & 1));
      if (early) request(j + 1);
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(w_ready + x * 2 + (j & 1));
      if (more && !early) {
        if (wait_all(s_bar(j + 1), ((j + 1) >> 1) & 1)) request(j + 1);
        else gave_up();
      }
    }
    tc::tmem_wait_ld();  // (after giving up, a request may be in flight)
    if (ok && !wait_all(o_done + x * 2 + ((n_tiles - 1) & 1), 0)) gave_up();
    if (ok) {
      tc::fence_after_sync();
      const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;
      const bool nans = *static_cast<volatile int*>(nan_any) != 0;
      // the warp's rows as bf16 in its part of the Q tile (no longer read), then
      // row by row to memory
#pragma unroll 1
      for (int ch = 0; ch < HD / 32; ++ch) {
        uint32_t ov[32];
        tc::tmem_ld32(o_tm(x) + lane_base + ch * 32, ov);
        tc::tmem_wait_ld();
        if (nans) {
          const volatile int* first = nan_s + ch * 32;
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (first[k] <= last) ov[k] = 0x7fc00000u;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[e] = pack_bf16x2(__uint_as_float(ov[8 * k + 2 * e]) * inv,
                               __uint_as_float(ov[8 * k + 2 * e + 1]) * inv);
          *reinterpret_cast<uint4*>(q_at(lane, ch * 4 + k)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      __syncwarp();
      const int first = job_s[0] + x * p.q_per_tile;  // the tile's first query
      const int nq = min(p.q_per_tile, job_s[1] - first);
      const int q_step = (p.n_heads - p.rep) * HD;
      __nv_bfloat16* tile_out =
          p.out + (int64_t(job_s[2] + first) * p.n_heads + job_s[3] * p.rep) * HD;
#pragma unroll 4
      for (int i = 0; i < STEPS; ++i) {
        const int m = i * RG + lane / RL;
        const int rr = (warp & 3) * 32 + m;
        const int q = (rr * p.rep_inv) >> 16;
        if (q < nq)
          reinterpret_cast<uint4*>(tile_out + int64_t(q) * q_step + rr * HD)[lane % RL] =
              *reinterpret_cast<const uint4*>(q_at(m, lane % RL));
      }
    }
  }
  // ------------------------------------------------------------ teardown
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int HD>
cudaError_t run_tc(const AttnArgs& a, const float* k_scales, const float* v_scales,
                   cudaStream_t stream) {
  using Lay = Layout<HD>;
  const PoolShape& pool = a.pool;
  const int rep = a.n_heads / pool.n_kv;
  TcParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k_pool = static_cast<const uint8_t*>(a.k_pool);
  p.v_pool = static_cast<const uint8_t*>(a.v_pool);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.err = a.err;
  p.n_heads = a.n_heads;
  p.n_kv = pool.n_kv;
  p.rep = rep;
  p.rep_inv = (65536 + rep - 1) / rep;  // (exact for rows < 128 of rep <= 16)
  p.W = a.max_blocks_per_seq;
  p.num_blocks = pool.num_blocks;
  p.max_len = a.max_seq_len;  // (no more than the tables hold)
  p.total_q = a.total_q;
  p.q_per_tile = kRows / rep;
  p.scale_log2 = a.scale * kLog2e;
  p.limits = ChunkLimits{a.total_q, a.max_q_len, a.max_seq_len,
                         int64_t(a.max_blocks_per_seq) * kBlk};
  auto kern = prefill_fp8_tc_kernel<HD>;
  static KernelSetup setup;
  cudaError_t e = kernel_setup(setup, kern, Lay::REQUEST, kThreads, nullptr);
  if (e != cudaSuccess) return e;
  const int qpp = 2 * p.q_per_tile;
  // ordered: one slot per (sequence, KV head, pair); the pairs number at most
  // total_q / qpp + one partial pair per sequence
  const int64_t slots = ((int64_t(a.total_q) + qpp - 1) / qpp + a.num_seqs) * pool.n_kv;
  p.ordered = a.num_seqs <= kThreads && slots <= INT_MAX;
  // natural order: the grid's z extent is 16-bit, so long batches go in slices
  const int slice = p.ordered ? a.num_seqs : 65535;
  for (int s0 = 0; s0 < a.num_seqs; s0 += slice) {
    p.B = std::min(slice, a.num_seqs - s0);
    p.bt = a.block_tables + int64_t(s0) * p.W;
    p.seq_lens = a.seq_lens + s0;
    p.cu_q = a.cu_q_lens + s0;
    p.last_seq = s0 + p.B == a.num_seqs ? p.B - 1 : -1;
    const dim3 grid = p.ordered ? dim3(static_cast<unsigned>(slots), 1, 1)
                                : dim3((a.max_q_len + qpp - 1) / qpp, pool.n_kv, p.B);
    if ((e = launch_pdl(kern, grid, kThreads, Lay::REQUEST, stream, p)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_prefill_fp8_tc(const AttnArgs& a, const float* k_scales, const float* v_scales,
                                  cudaStream_t stream) {
  return a.pool.head_dim == 64 ? run_tc<64>(a, k_scales, v_scales, stream)
                               : run_tc<128>(a, k_scales, v_scales, stream);
}

}  // namespace pkv
