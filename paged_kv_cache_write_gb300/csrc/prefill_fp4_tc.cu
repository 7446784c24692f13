// Chunked prefill over the 4-bit cache on the 5th-generation tensor cores: bf16
// queries, head_dim 64 / 128.
//
// What is computed: query i of a chunk of c queries at the end of an L-token sequence
// attends keys 0 .. L - c + i of its KV head, with element = code x group scale x head
// scale.  With k4, v4 the products of code and group scale, kg, vg the head's scales:
//   x = (q . k4) * (scale * log2 e * kg),  w = 2^(x - M + 4),
//   l += sum of w,  O += w v4,  out = vg O / l.
// M is a running reference of x, moved to the maximum when a weight would pass f16's
// 65,504 (the maximum has grown 2^12-fold: seldom after the first tile; f16 is normal
// down to 2^-18 of the reference's weight).
//
// tcgen05 takes 4-bit operands only beside others of at most 8 bits, which would cost
// the queries and weights their precision, so codes times group scales become f16
// (exact) on their way into shared memory.  Queries become f16 too, each row times the
// power of two that brings its largest element to 2^14 .. 2^15 (exact for bf16 within
// 2^28 of it; undone in the score's factor).
//
// A job is two 128-row tiles, A and B, of one (sequence, KV head); a row is one (query,
// query head) pair.  A grid has a CTA for every job, but one CTA per SM goes on: before it
// ends a job it takes over a CTA that has not started (clusterlaunchcontrol), so that the
// order of the batch is found once, and the next job's keys, values and queries are on
// their way while the last one's softmax ends, yet the GPU still hands out the jobs one by
// one.  (A CTA for each job: 64 prompts of 64 tokens of 32 heads on 8 of 64 28.6 us, now
// 23.2; 32 of 256 52.6, now 44.5; 32 of 128 - 2,048 482, now 419.  Jobs dealt out in turn
// instead: 538 us for the last.)
//
// Keys go in tiles of 64 (4 blocks), so that scores have two buffers per row tile in TMEM:
// while a tile's softmax runs, its next scores are computed, and neither waits for the
// other.
//  warps 0-3    softmax of tile A, 4-7 of tile B: one thread per row.  Weights are
//               computed against the reference as it stands; only if some weight came
//               out past f16's range (their partial sums tell) the maximum is taken,
//               the reference moved to it and the tile done again, so that most tiles
//               need no maximum at all.  Weights go back to TMEM as f16 over the
//               scores.
//  warps 8, 9   issue the MMAs of tiles A and B, one elected lane each: S_X of the
//               first two key tiles, then for each key tile j, once its weights are
//               there, O_X += W_X V_j and S_X = Q_X K_{j+2}^T.  Warp 8 allocates TMEM:
//               2 S_A, 2 S_B, O_A, O_B, all 512 columns at head_dim 128.
//  warps 10-15  bring K and V, a block (16 tokens) at a time in turn: 16-byte loads
//               straight from the pool, where a head's rows of a block lie together,
//               each warp's next blocks on their way, codes -> f16 in registers,
//               128-byte-swizzled tiles in four-stage rings.  Warp 10 finds the jobs.
//
// Bound by the softmax warps: 1,640 cycles a key tile, of which exponentials and
// conversions alone are 1,000 (the MMAs: 1,330 at head_dim 128), and what a job adds, some
// 7,000 at 64 and 12,000 at 128 (queries in, first scores, outputs).  64 heads on 8 of 128,
// 4 chunks of 512 after 990 - 3,018 tokens: 142.5 - 145 us, 1,026 TFLOP/s at the least; 2 chunks of 1,024 that
// end at 4,096 tokens 223 us, 1,080.  32 heads on 8 of 64, whole prompts: 2 of 4,096 tokens
// 228 us, 603; 32 of 256 195.
//
// Two row tiles a CTA, because they share the conversion of K and V, and one CTA an SM:
// CTAs of one row tile, two on an SM, hide each other's start and end but took 28% longer
// for 8 chunks of 1,024 of 32 heads on 8 of 64, 10% for 30 prompts of 33 - 612 tokens.
//
// 16 warps leave 128 registers a thread, and a loop that spills pays for it: with 200 KB of
// shared memory little L1 is left, and a reload from local memory costs an L2 round trip.
// (For heads of 128 a thread stores 8 bytes there and reads 16, for 64 none.)
//
// Output sums stay in TMEM over the whole sequence.  The tensor cores cut them off: an
// output is too small by some 2^-23 for every 16 keys, 6.5e-4 over 131,072.
//
// Values past the sequence's end are stored as zeros (scales taken as zero).  A group
// of values under a NaN scale that some row of the tile may not see is stored as zeros
// too, and its first position noted: rows that do see it get NaN at the end.  Every
// wait is bounded; a thread that gave up still takes part in the CTA's barriers.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "device.cuh"
#include "fp4.cuh"
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
constexpr int kTiles = 2;    // row tiles of a CTA
constexpr int kMmaWarp = 8;  // and 9, after eight of the softmax
constexpr int kLoadWarp0 = 10;
constexpr int kLoadWarps = 6;
constexpr int kAhead = 3;  // blocks in flight per load warp
constexpr int kThreads = 16 * 32;
constexpr uint32_t kTmemCols = 512;
constexpr int kStages = 4;
constexpr int kJobs = 16;  // places of jobs: more than the roles can be apart (load warps)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kWeightLog2 = 4.f;     // log2 of the reference's weight
constexpr float kWeightMax = 65504.f;  // f16's largest

struct TcParams {
  const __nv_bfloat16* q;
  const uint8_t *k_pool, *v_pool, *k_groups, *v_groups;
  const float *k_scale, *v_scale;
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
  static constexpr int K_OFF = kTiles * Q_TILE;  // after Q_A, Q_B
  static constexpr int V_OFF = K_OFF + kStages * KV_TILE;
  static constexpr int NG = HD / 16;                    // groups of a row
  static constexpr int NAN_OFF = V_OFF + kStages * KV_TILE;  // [kJobs][NG + 1]
  static constexpr int BAR_OFF = (NAN_OFF + kJobs * (NG + 1) * 4 + 15) / 16 * 16;
  static constexpr int JOB_OFF = BAR_OFF + 512;      // [kJobs]
  static constexpr int TAB_OFF = JOB_OFF + kJobs * 32;  // [5][kThreads] + 1: the batch in its order
  static constexpr int BYTES = TAB_OFF + 5 * kThreads * 4 + 16;
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

// Takes the next CTA of the grid that has not started: its index, if there is one, comes to
// the 16 bytes at `to`, with 16 bytes on the barrier.
__device__ __forceinline__ void try_cancel(void* to, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_addr(to)),
      "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ bool cancelled(const void* at, dim3& cta) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 lo, hi;\n\t.reg .b128 h;\n\t"
      "ld.shared.v2.b64 {lo, hi}, [%4];\n\t"
      "mov.b128 h, {lo, hi};\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, %2, %3, _}, h;\n\t}"
      : "=r"(ok), "=r"(cta.x), "=r"(cta.y), "=r"(cta.z)
      : "r"(smem_addr(at))
      : "memory");
  return ok != 0;
}

// What a CTA works on: a group of row tiles of a sequence and KV head.
struct alignas(16) Job {
  int tiles;             // of keys; 0: no more jobs
  int b, g, i0, q0, c, L;  // sequence, KV head, first query; the sequence's rows and keys
  int pad;
};
static_assert(sizeof(Job) == 32, "the places below");

template <int HD>
__global__ void __launch_bounds__(kThreads, 1) prefill_fp4_tc_kernel(const TcParams p) {
  using Lay = Layout<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);

  asm volatile("griddepcontrol.wait;" ::: "memory");  // the preceding kernel's results
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
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
  uint64_t* job_full = bars + 32;      // [kJobs]
  uint64_t* next_bar = bars + 32 + kJobs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(next_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* next_s = reinterpret_cast<uint8_t*>(bars) + 496;  // [16] (bars are 16-byte aligned)
  static_assert((32 + kJobs + 2) * 8 <= 496, "barriers");
  Job* jobs = reinterpret_cast<Job*>(smem + Lay::JOB_OFF);
  int* nan_s = reinterpret_cast<int*>(smem + Lay::NAN_OFF);  // [job % kJobs][NG first positions, flag]

  // Work order, as in the bf16 prefill: with at most blockDim.x sequences, the grid's CTAs
  // are the (sequence, KV head, group of row tiles) triples, sequences by descending work
  // and each one's groups from the last (most keys) down; otherwise x, y, z are group, KV
  // head and sequence.  Work values are staged in the (still unused) V stages.  What needs
  // no sequence is set up while their offsets and lengths come.
  int* at_s = reinterpret_cast<int*>(smem + Lay::TAB_OFF);  // by sequence: offsets, lengths
  int* end_s = at_s + kThreads;
  int* len_s = end_s + kThreads;
  int* seq_s = len_s + kThreads;     // by rank: the sequence, its first group
  int* first_s = seq_s + kThreads;   // [B + 1]
  const int qpg = kTiles * p.q_per_tile;  // queries of a group
  const int t = threadIdx.x;
  int at = 0, end = 0, len = 0;
  if (p.ordered && t < p.B) {
    at = p.cu_q[t];
    end = p.cu_q[t + 1];
    len = p.seq_lens[t];
  }
  if (t == 32) {
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(q_full + i, 4);
      mbar_init(drain + i, 1);
    }
    for (int i = 0; i < 2 * kTiles; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(w_ready + i, 4);
      mbar_init(o_done + i, 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(k_full + i, kBlocks);
      mbar_init(k_empty + i, kTiles);  // left by the row tiles
      mbar_init(v_full + i, kBlocks);
      mbar_init(v_empty + i, kTiles);
    }
    for (int i = 0; i < kJobs; ++i) mbar_init(job_full + i, 1);
    mbar_init(next_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    if (p.ordered) mbar_arrive(job_full);  // (the CTA's own job is written below)
  }
  auto nan_of = [&](int job) { return nan_s + (job % kJobs) * (Lay::NG + 1); };
  auto clear_nan = [&](int* n, int i) { n[i] = i < Lay::NG ? INT_MAX : 0; };
  if (t >= 64 && t < 64 + kJobs)
    for (int i = 0; i <= Lay::NG; ++i) clear_nan(nan_of(t - 64), i);
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  // Fills in a job; whether there is something to do: a chunk within the rows, no longer
  // than its sequence, and queries in the group.
  auto fill = [&](Job& o, int b, int g, int i0, int q0, int end, int len) {
    o.b = b;
    o.g = g;
    o.i0 = i0;
    o.q0 = q0;
    o.c = end - q0;
    o.L = min(len, p.max_len);
    if (q0 < 0 || end <= q0 || end > p.total_q || o.L < o.c || i0 < 0 || i0 >= o.c) return false;
    o.tiles = (o.L - o.c + min(o.c, i0 + qpg) - 1) / kTileKeys + 1;
    return true;
  };
  if (p.ordered) {
    int64_t* work_s = reinterpret_cast<int64_t*>(smem + Lay::V_OFF);
    int* groups_s = reinterpret_cast<int*>(work_s + p.B);
    if (t < p.B) {
      if (blockIdx.x == 0) report_bad_chunk(p.err, p.limits, at, end, len, t == p.last_seq);
      Job o;
      const bool any = fill(o, t, 0, 0, at, end, len);
      work_s[t] = any ? int64_t(o.c) * (2 * int64_t(o.L) - o.c + 1) : 0;
      groups_s[t] = any ? (o.c - 1) / qpg + 1 : 0;
      at_s[t] = at;
      end_s[t] = end;
      len_s[t] = len;
    }
    if (t == 0) jobs[0].tiles = 0;
    __syncthreads();
    // a sequence's rank and first group: the heavier ones' number and groups, summed by
    // several threads for each sequence
    int share = 1;
    while (share < 32 && 2 * share * p.B <= kThreads) share *= 2;
    const int mine = t / share, part = t & (share - 1);
    int64_t first = 0;
    int rank = 0;
    if (mine < p.B) {
      const int64_t wt = work_s[mine];
#pragma unroll 4
      for (int i = part; i < p.B; i += share) {
        const int64_t wi = work_s[i];
        if (wi > wt || (wi == wt && i < mine)) first += groups_s[i], ++rank;
      }
    }
    for (int o = 1; o < share; o <<= 1) {
      first += __shfl_xor_sync(0xffffffffu, first, o);
      rank += __shfl_xor_sync(0xffffffffu, rank, o);
    }
    if (mine < p.B && part == 0) {
      seq_s[rank] = mine;
      first_s[rank] = static_cast<int>(min(first, int64_t(INT_MAX)));
      const int groups = groups_s[mine];
      if (rank == p.B - 1) first_s[p.B] = static_cast<int>(min(first + groups, int64_t(INT_MAX)));
      const int64_t off = blockIdx.x - first * p.n_kv;
      if (off >= 0 && off < int64_t(groups) * p.n_kv) {
        const int o = static_cast<int>(off), g = o / groups;
        fill(jobs[0], mine, g, (groups - 1 - (o - g * groups)) * qpg, at_s[mine], end_s[mine],
             len_s[mine]);
      }
    }
  } else if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
    for (int b = t; b < p.B; b += kThreads)
      report_bad_chunk(p.err, p.limits, p.cu_q[b], p.cu_q[b + 1], p.seq_lens[b], b == p.last_seq);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  // 1: the CTA's job is in `o`; 0: it has none; -1: nor have the ones after it
  auto find_job = [&](dim3 cta, Job& o) -> int {
    if (!p.ordered) {
      const int b = static_cast<int>(cta.z);
      return fill(o, b, cta.y, cta.x * qpg, p.cu_q[b], p.cu_q[b + 1], p.seq_lens[b]);
    }
    const int xg = static_cast<int>(cta.x / static_cast<uint32_t>(p.n_kv));
    if (xg >= first_s[p.B]) return -1;
    int r = 0, n = p.B;  // the last rank whose first group is not past xg
    while (n > 1) {
      const int h = n >> 1;
      if (first_s[r + h] <= xg) r += h, n -= h;
      else n = h;
    }
    const int groups = first_s[r + 1] - first_s[r], b = seq_s[r];
    const int off = static_cast<int>(cta.x) - first_s[r] * p.n_kv, g = off / groups;
    return fill(o, b, g, (groups - 1 - (off - g * groups)) * qpg, at_s[b], end_s[b], len_s[b]);
  };
  // every wait is one of these two: bounded, by a whole warp or by one lane
  auto wait_one = [&](uint64_t* bar, uint32_t parity) {
    return wait_or_abort(bar, parity, abort_flag);
  };
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    return warp_wait_or_abort(bar, parity, abort_flag);
  };
  auto q_tile = [&](int x) { return smem + x * Lay::Q_TILE; };
  auto k_st = [&](int j) { return smem + Lay::K_OFF + (j % kStages) * Lay::KV_TILE; };
  auto v_st = [&](int j) { return smem + Lay::V_OFF + (j % kStages) * Lay::KV_TILE; };
  auto s_tm = [&](int x, int j) { return tmem + uint32_t(x * 2 + (j & 1)) * kTileKeys; };
  auto o_tm = [&](int x) { return tmem + uint32_t(kTiles + x) * 128u; };

  if (warp >= kLoadWarp0) {
    // ------------------------------------------------------ K and V tiles
    // Unit 8 j + i is block i of K tile j, unit 8 j + 4 + i of V tile j; the warps take
    // them in turn.  Lane: 16-byte piece (32 dims) lane % PR of row lane / PR, in steps
    // of RS rows.  A piece is four 16-byte pieces of f16, one from each word; at
    // head_dim 128 the lanes of a row's second half take their words in another order,
    // so that the eight lanes of a store phase touch each bank once.
    constexpr int PR = HD / 32;    // pieces of a row
    constexpr int RS = 32 / PR;    // rows per step: 8 or 16
    constexpr int NV = kBlk / RS;  // steps: 2 or 1
    const int piece = lane % PR, half = piece >> 1;
    const int r0 = lane / PR;  // row of step 0
    // where word q of the lane's piece goes in row r0 + RS i of a block: (r0 + RS i) % 8
    // is r0 % 8
    const int turn = HD == 128 && half ? 2 : 0;
    const int put = half * Lay::KV_HALF + r0 * 128;
    const int unit0 = (piece & 1) * 4;
    const int w = warp - kLoadWarp0;
    bool ok = true;
    auto gave_up = [&]() {
      if (lane == 0) {
        report(p.err, PKV_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      ok = false;
    };
    // The roles count jobs, and key tiles over all of them: stages and buffers go on from
    // job to job.  This warp 0 finds the jobs: the CTA's own first, then those of CTAs that
    // have not started, which it takes over one at a time.  (After some without work, which
    // only the natural order has, it leaves the rest to the GPU, and the CTA ends: the
    // others do not wait for long.)
    uint32_t takes = 0;
    auto next_job = [&](int job) {  // lane 0
      Job o;
      o.tiles = 0;
      int what = job == 0 ? find_job(blockIdx, o) : 0;
      for (int tries = 0; what == 0 && tries < 32; ++tries) {
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(next_bar, 16);
        try_cancel(next_s, next_bar);
        // (not given up for others' sake: it is on its way here)
        bool there = false;
        for (uint32_t i = 0; i < kFp8Polls && !there; ++i) there = mbar_park(next_bar, takes & 1);
        ++takes;
        dim3 cta;
        if (!there) {
          report(p.err, PKV_DEVERR_TIMEOUT);
          *abort_flag = 1;
          what = -1;
        } else {
          what = cancelled(next_s, cta) ? find_job(cta, o) : -1;
        }
      }
      if (what <= 0) o.tiles = 0;
      jobs[job % kJobs] = o;
      mbar_arrive(job_full + job % kJobs);
    };
    for (int job = 0, t0 = 0; ok; ++job) {
      // (a job only once tile A's softmax has come to the one before: not further ahead, so
      // that CTAs end at about the same time)
      if (w == 0) {
        if (job > 0 && !wait_all(q_full, (job - 1) & 1)) {
          gave_up();
          break;
        }
        if (lane == 0 && (job > 0 || !p.ordered)) next_job(job);
        __syncwarp();
      }
      if (!wait_all(job_full + job % kJobs, (job / kJobs) & 1)) {
        gave_up();
        break;
      }
      const Job& o = jobs[job % kJobs];
      const int n_tiles = o.tiles;
      if (n_tiles == 0) break;
      const int b = o.b, g = o.g, i0 = o.i0, c = o.c, L = o.L;
      const int n_blocks_seq = (L + kBlk - 1) / kBlk;
      if (job > 0) {
        // the queries into L2, which the softmax will ask for when the job before has ended
        // (heads of 128, 32 prompts of 256 tokens: 144 -> 126 us)
        const int lines = p.rep * HD / 64;  // a query's, of 128 bytes
        const int n = min(qpg, c - i0) * lines;
        const __nv_bfloat16* q = p.q + (int64_t(o.q0 + i0) * p.n_heads + g * p.rep) * HD;
        for (int e = w * 32 + lane; e < n; e += kLoadWarps * 32) {
          const int qi = e / lines;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q + int64_t(qi) * p.n_heads * HD + (e - qi * lines) * 64));
        }
      }
      const int32_t* row = p.bt + int64_t(b) * p.W;
      const int n_units = 2 * kBlocks * n_tiles;
      // The place of the job eight on, and eight back.  That one's softmax has ended: this
      // warp has stored blocks of the last job's last tile, in a stage that tile T - 4 has
      // left, whose scores came after the softmax of T - 6 or of the whole job before; and a
      // job has a tile or more.  No load warp has values of that one yet: V tile T + 4 waits
      // for tile T, of which this warp has a block to bring.
      if (w == 0 && lane <= Lay::NG) clear_nan(nan_of(job + kJobs / 2), lane);
      int* nan_j = nan_of(job);
      // -1: the sequence has no block there
      auto id_of = [&](int u) {
        const int jb = (u >> 3) * kBlocks + (u & 3);
        int id = -1;
        if (u < n_units && jb < n_blocks_seq) id = row[jb];
        return id;
      };
      uint4 d[kAhead][NV];
      uint32_t ds[kAhead][NV];  // the scales of a piece's two groups
      int id_d[kAhead], id_next[kAhead];
      // (unconditional loads, of block 0 where there is none, so that they stay in flight:
      // a selected load is waited for where it is issued)
      auto fetch = [&](uint4 (&x)[NV], uint32_t (&sx)[NV], int& id, int u) {
        if (id >= p.num_blocks || id < 0) id = -1;
        const int64_t first = (int64_t(max(id, 0)) * p.n_kv + g) * kBlk + r0;
        const uint8_t* src = ((u & 4) ? p.v_pool : p.k_pool) + first * (HD / 2) + piece * 16;
        const uint8_t* grp = ((u & 4) ? p.v_groups : p.k_groups) + first * Lay::NG + piece * 2;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          x[i] = *reinterpret_cast<const uint4*>(src + i * RS * (HD / 2));
          sx[i] = *reinterpret_cast<const uint16_t*>(grp + i * RS * Lay::NG);
        }
      };
      // (unit 8 T of the CTA's tile T goes to warp 8 T % 6)
      const int w0 = (w + 6 - (8 * (t0 % 3)) % 6) % 6;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int u = w0 + k * kLoadWarps;
        id_d[k] = id_of(u);
        fetch(d[k], ds[k], id_d[k], u);
        id_next[k] = id_of(u + kAhead * kLoadWarps);
      }
      for (int u0 = w0; u0 < n_units && ok; u0 += kAhead * kLoadWarps) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int u = u0 + k * kLoadWarps;
          if (u >= n_units || !ok) break;
          const int j = u >> 3, bi = u & 3;
          const bool is_v = (u & 4) != 0;
          const int st = (t0 + j) % kStages;
          const uint32_t use = (t0 + j) / kStages;
          if (use > 0 && !wait_all((is_v ? v_empty : k_empty) + st, (use - 1) & 1)) {
            gave_up();
            break;
          }
          const int pos0 = (j * kBlocks + bi) * kBlk;
          if (!is_v && lane == 0 && id_d[k] < 0 && pos0 < L)
            report(p.err, PKV_DEVERR_BLOCK_ID);  // (a block that it holds)
          if (id_d[k] < 0 || pos0 + kBlk > L) {
            // what lies past the sequence's end, and a bad block, is zeros
#pragma unroll
            for (int i = 0; i < NV; ++i)
              if (id_d[k] < 0 || pos0 + r0 + RS * i >= L) ds[k][i] = 0u;
          }
          if (is_v && pos0 + kBlk > L - c + i0 + 1) {
            // some row may not see some key of this block: take out its NaNs
            const int first_last = L - c + i0;  // the last key that the pair's first query sees
#pragma unroll
            for (int i = 0; i < NV; ++i) {
              const int pos = pos0 + r0 + RS * i;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if (((ds[k][i] >> (8 * e)) & 0x7fu) == 0x7fu && pos > first_last) {
                  atomicMin(nan_j + piece * 2 + e, pos);
                  atomicOr(nan_j + Lay::NG, 1);
                  ds[k][i] &= ~(0xffu << (8 * e));
                }
              }
            }
          }
          uint8_t* base = (is_v ? v_st(t0 + j) : k_st(t0 + j)) + bi * (kBlk * 128) + put;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            // words and scales in the lane's order
            const uint4 x = d[k][i];
            const uint32_t wd[4] = {turn ? x.z : x.x, turn ? x.w : x.y, turn ? x.x : x.z,
                                    turn ? x.y : x.w};
            const uint32_t s2 = e4m3x2_to_f16x2(static_cast<uint16_t>(ds[k][i]));
            const uint32_t sc[2] = {__byte_perm(s2, s2, turn ? 0x3232 : 0x1010),
                                    __byte_perm(s2, s2, turn ? 0x1010 : 0x3232)};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t f[4];
              fp4::codes_to_f16x2(wd[q], f);
#pragma unroll
              for (int e = 0; e < 4; ++e) f[e] = fp4::mul_f16x2(f[e], sc[q >> 1]);
              // 16-byte piece n of row r sits at n ^ (r % 8)
              const int n = unit0 + (q ^ turn);
              *reinterpret_cast<uint4*>(base + i * RS * 128 + ((n ^ (r0 & 7)) << 4)) =
                  make_uint4(f[0], f[1], f[2], f[3]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive((is_v ? v_full : k_full) + st);
          const int un = u + kAhead * kLoadWarps;
          id_d[k] = id_next[k];
          fetch(d[k], ds[k], id_d[k], un);
          id_next[k] = id_of(un + kAhead * kLoadWarps);
        }
      }
      t0 += n_tiles;
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
      auto issue_pv = [&](int x, int j, bool more) {  // more: added to what is there
        const uint64_t vd = v_desc + uint32_t((j % kStages) * Lay::KV_TILE) / 16;
#pragma unroll
        for (int kk = 0; kk < kTileKeys / 16; ++kk)
          // W: 16 f16 are 8 columns
          tc::mma_ts(o_tm(x), s_tm(x, j) + kk * 8, vd + kk * 2048 / 16, idesc_pv, more || kk > 0);
      };
      const int x = warp - kMmaWarp;
      bool ok = true;
      for (int job = 0, t0 = 0; ok; ++job) {
        if (!(ok = wait_one(job_full + job % kJobs, (job / kJobs) & 1))) break;
        const int n_tiles = jobs[job % kJobs].tiles;
        if (n_tiles == 0) break;
        // (the row tile's last scores have been taken, and its weights multiplied, in order)
        ok = wait_one(q_full + x, job & 1);
        for (int j = 0; j < 2 && j < n_tiles && ok; ++j) {
          const int T = t0 + j;
          if (!(ok = wait_one(k_full + T % kStages, (T / kStages) & 1))) break;
          tc::fence_after_sync();
          issue_qk(x, T);
          tc::commit(k_empty + T % kStages);  // this row tile has read K_j
        }
        for (int j = 0; j < n_tiles && ok; ++j) {
          const int T = t0 + j, st = T % kStages, kn = (T + 2) % kStages;
          const bool more = j + 2 < n_tiles;
          // (the weights last: once they are there both products go at once)
          ok = wait_one(v_full + st, (T / kStages) & 1) &&
               (!more || wait_one(k_full + kn, ((T + 2) / kStages) & 1)) &&
               wait_one(w_ready + x * 2 + (T & 1), (T >> 1) & 1);
          if (!ok) break;
          tc::fence_after_sync();
          issue_pv(x, T, j > 0);
          tc::commit(o_done + x * 2 + (T & 1));
          tc::commit(v_empty + st);
          if (!more) continue;
          issue_qk(x, T + 2);
          tc::commit(k_empty + kn);
        }
        t0 += n_tiles;
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
    // A row's 16-byte vectors of q (and of out) are RL = HD / 8 lanes' work: the warp goes
    // through its rows 32 / RL at a time, so that memory is touched row by row (with every
    // lane at a row of its own, 32 lines a load, one tile of 64 tokens took 3 us longer).
    // What says whose row it is is read from shared memory where it is needed, so that it
    // takes no registers in between.
    constexpr int RL = HD / 8, RG = 32 / RL, STEPS = 32 / RG;
    // where vector k of row m of the warp lies in the Q tile
    auto q_at = [&](int m, int k) {
      const int rr = (warp & 3) * 32 + m;
      return q_tile(x) + (k >> 3) * Lay::Q_HALF + rr * 128 + (((k & 7) ^ (rr & 7)) << 4);
    };
    bool ok = true;
    auto gave_up = [&]() {
      if (lane == 0) {
        report(p.err, PKV_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      ok = false;
    };
    for (int job = 0, t0 = 0; ok; ++job) {
      if (!wait_all(job_full + job % kJobs, (job / kJobs) & 1)) {
        gave_up();
        break;
      }
      const Job& o = jobs[job % kJobs];
      const int n_tiles = o.tiles;
      if (n_tiles == 0) break;
      int last, cut;   // last key that the row sees; the least of the warp's rows
      float rs = 1.f;  // undoes the row's power of two; times the score's factor
      const float factor = p.scale_log2 * p.k_scale[o.g];
      {
        // every row's vectors on their way at once
        const int tile_first = o.i0 + x * p.q_per_tile;  // the tile's first query
        const int nq = min(p.q_per_tile, o.c - tile_first);
        const int q_step = (p.n_heads - p.rep) * HD;
        const __nv_bfloat16* tile_q =
            p.q + (int64_t(o.q0 + tile_first) * p.n_heads + o.g * p.rep) * HD;
        {
          const int q = (((warp & 3) * 32 + lane) * p.rep_inv) >> 16;  // row / rep
          last = q < nq ? o.L - o.c + tile_first + q : INT_MAX;  // a row without a query is never masked
          cut = __reduce_min_sync(0xffffffffu, last);
        }
        uint4 u[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          const int rr = (warp & 3) * 32 + i * RG + lane / RL;
          const int q = (rr * p.rep_inv) >> 16;
          u[i] = make_uint4(0u, 0u, 0u, 0u);
          if (q < nq) u[i] = reinterpret_cast<const uint4*>(tile_q + int64_t(q) * q_step + rr * HD)[lane % RL];
        }
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          const uint32_t e[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
          // the row's largest magnitude
          __nv_bfloat162 m2 = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&e[0]));
#pragma unroll
          for (int k = 1; k < 4; ++k)
            m2 = __hmax2(m2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&e[k])));
#pragma unroll
          for (int o = 1; o < RL; o <<= 1) m2 = __hmax2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
          const float a = fmaxf(__low2float(m2), __high2float(m2));
          const int up = min(126, 14 + 127 - static_cast<int>(__float_as_uint(a) >> 23));
          const float f = pow2f(up);
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            o[k] = pack_f16x2(__uint_as_float(e[k] << 16) * f,
                              __uint_as_float(e[k] & 0xffff0000u) * f);
          *reinterpret_cast<uint4*>(q_at(i * RG + lane / RL, lane % RL)) =
              make_uint4(o[0], o[1], o[2], o[3]);
          // the factor goes to the lane whose row it is
          const float back = __shfl_sync(0xffffffffu, pow2f(-up), (lane % RG) * RL);
          if (lane / RG == i) rs = back * factor;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full + x);
      }
      rs = fmaxf(rs, 1.2e-38f);  // (not zero: -inf stays -inf)
      float m_used = -INFINITY, l_sum = 0.f;
      uint32_t v[kTileKeys];  // scores
      auto request = [&](int j) {  // (there after tmem_wait_ld)
        tc::fence_after_sync();
        tc::tmem_ld32(s_tm(x, j) + lane_base, *reinterpret_cast<uint32_t(*)[32]>(v));
        tc::tmem_ld32(s_tm(x, j) + lane_base + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
      };
      auto s_bar = [&](int T) { return s_full + x * 2 + (T & 1); };
      if (wait_all(s_bar(t0), (t0 >> 1) & 1)) request(t0);
      else gave_up();
      for (int j = 0; j < n_tiles && ok; ++j) {
        const int T = t0 + j;
        const uint32_t s_addr = s_tm(x, T) + lane_base;
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
            float mx = __uint_as_float(v[0]);
#pragma unroll
            for (int k = 1; k < kTileKeys; ++k) mx = fmaxf(mx, __uint_as_float(v[k]));
            mx *= rs;
            const float m_new = fmaxf(m_used, mx);
            if (m_new > m_used) d = m_used - m_new;
            m_used = m_new;
          }
          rescale = pass > 0;
          const float mref = (m_used == -INFINITY ? 0.f : m_used) - kWeightLog2;
          const float2 f2 = make_float2(rs, rs), c2 = make_float2(-mref, -mref);
          float most = 0.f;
          add = 0.f;
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            uint32_t pk[16];
#pragma unroll
            for (int bb = 0; bb < 2; ++bb) {
              const int bk = ch * 2 + bb;
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
              add += acc.x + acc.y;
              most = fmaxf(most, fmaxf(acc.x, acc.y));  // no weight is larger
            }
            tc::tmem_st16(s_addr + ch * 16, pk);
          }
          move = most > kWeightMax;
          if (!__any_sync(0xffffffffu, move)) break;
          tc::tmem_wait_st();  // the second pass stores to the same columns
        }
        l_sum = l_sum * fast_exp2(d) + add;
        if (rescale && j > 0) {
          // O_X has to hold all products before this tile's.  S_{j+1} was computed
          // after them; only the last tiles have a barrier for it of their own.
          // (W_j is not there yet, so no later phase can have completed.)
          const bool there =
              j + 1 < n_tiles ? wait_all(s_bar(T + 1), ((T + 1) >> 1) & 1)
                              : wait_all(o_done + x * 2 + ((T - 1) & 1), ((T - 1) >> 1) & 1);
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
            more && __all_sync(0xffffffffu, mbar_test(s_bar(T + 1), ((T + 1) >> 1) & 1));
        if (early) request(T + 1);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(w_ready + x * 2 + (T & 1));
        if (more && !early) {
          if (wait_all(s_bar(T + 1), ((T + 1) >> 1) & 1)) request(T + 1);
          else gave_up();
        }
      }
      tc::tmem_wait_ld();  // (after giving up, a request may be in flight)
      const int end_tile = t0 + n_tiles - 1;
      if (ok && !wait_all(o_done + x * 2 + (end_tile & 1), (end_tile >> 1) & 1)) gave_up();
      if (ok) {
        tc::fence_after_sync();
        const float inv = l_sum == 0.f ? 0.f : p.v_scale[o.g] / l_sum;
        const volatile int* nan_j = nan_of(job);
        const bool nans = nan_j[Lay::NG] != 0;
        // the warp's rows as bf16 in its part of the Q tile (no longer read), then
        // row by row to memory
#pragma unroll 1
        for (int ch = 0; ch < HD / 32; ++ch) {
          uint32_t ov[32];
          tc::tmem_ld32(o_tm(x) + lane_base + ch * 32, ov);
          tc::tmem_wait_ld();
          if (nans) {
            const volatile int* first = nan_j + ch * 2;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (first[k / 16] <= last) ov[k] = 0x7fc00000u;
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
        const int first = o.i0 + x * p.q_per_tile;  // the tile's first query
        const int nq = min(p.q_per_tile, o.c - first);
        const int q_step = (p.n_heads - p.rep) * HD;
        __nv_bfloat16* tile_out =
            p.out + (int64_t(o.q0 + first) * p.n_heads + o.g * p.rep) * HD;
#pragma unroll 4
        for (int i = 0; i < STEPS; ++i) {
          const int m = i * RG + lane / RL;
          const int rr = (warp & 3) * 32 + m;
          const int q = (rr * p.rep_inv) >> 16;
          if (q < nq)
            reinterpret_cast<uint4*>(tile_out + int64_t(q) * q_step + rr * HD)[lane % RL] =
                *reinterpret_cast<const uint4*>(q_at(m, lane % RL));
        }
        __syncwarp();  // (the next job's queries go where these rows lay)
        tc::fence_before_sync();
      }
      t0 += n_tiles;
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
cudaError_t run_tc(const AttnArgs& a, const Fp4Cache& cache, cudaStream_t stream) {
  using Lay = Layout<HD>;
  const PoolShape& pool = a.pool;
  const int rep = a.n_heads / pool.n_kv;
  TcParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k_pool = static_cast<const uint8_t*>(cache.k_pool);
  p.v_pool = static_cast<const uint8_t*>(cache.v_pool);
  p.k_groups = static_cast<const uint8_t*>(cache.k_groups);
  p.v_groups = static_cast<const uint8_t*>(cache.v_groups);
  p.k_scale = cache.k_scale;
  p.v_scale = cache.v_scale;
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
  auto kern = prefill_fp4_tc_kernel<HD>;
  static KernelSetup setup;
  cudaError_t e = kernel_setup(setup, kern, Lay::REQUEST, kThreads, nullptr);
  if (e != cudaSuccess) return e;
  const int qpg = kTiles * p.q_per_tile;
  // ordered: one slot per (sequence, KV head, group of row tiles); the groups number at
  // most total_q / qpg + one partial group per sequence
  const int64_t slots = ((int64_t(a.total_q) + qpg - 1) / qpg + a.num_seqs) * pool.n_kv;
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
                                : dim3((a.max_q_len + qpg - 1) / qpg, pool.n_kv, p.B);
    if ((e = launch_pdl(kern, grid, kThreads, Lay::REQUEST, stream, p)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_prefill_fp4_tc(const AttnArgs& a, const Fp4Cache& c, cudaStream_t stream) {
  return a.pool.head_dim == 64 ? run_tc<64>(a, c, stream) : run_tc<128>(a, c, stream);
}

}  // namespace pkv
