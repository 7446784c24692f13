// Decode over the 8-bit cache: one query per sequence attends to the
// sequence's pages (attention.cuh's decode over e4m3 pools with a scale per
// block and KV head; mathematics and layouts of the tiles in fp8_rows.cuh).
//
// Bound by reading the cache: 2 x n_kv x head_dim bytes a token, 8 bytes of
// scales per block and head.  The work split is that of the bf16 decode, since
// what it is for is the same: a persistent grid over equal contiguous ranges
// of (sequence, head group, block) units, a joining kernel for the groups that
// several CTAs share, and one thread-block cluster per (sequence, head group)
// for batches too small to stream.  A producer lane fetches whole blocks of the
// group's heads with TMA (16 tokens x hg heads x head_dim bytes, K and V: 32 KB
// a stage at 8 heads of 128); one consumer warp per KV head.  Block ids and
// scales are gathered by the consumer warps, 32 blocks at a time and a batch
// ahead of use, so their latency is off the path.
//
// Measured, bf16 queries, where a plain copy reaches 6.79 TB/s: 256 sequences
// of 2,040 - 2,048 tokens, 8 KV heads: head_dim 128 163 us (6.6 TB/s), 64 87 us
// (6.2 TB/s), 32 58 us (4.7 TB/s), 16 51 us (2.7 TB/s: the consumers' chains, the
// same for any width, bound narrow heads).  64 sequences of 512 - 2,048 tokens
// of 8 x 64 (81 MB) 23 us, of which 12 stream; the rest is the plan (2 us),
// the first scales and tile (2 us) and the joining launch (3 us, 1.2 of which an
// empty one would take too).
#pragma once

#include "attention.cuh"
#include "fp8_rows.cuh"

namespace pkv {
namespace fp8 {

using attn::DecodeParams;
using attn::DecodeWs;
using attn::Ring;
using attn::kBarrierBytes;
using attn::kKernelPlanSeqs;
using attn::kMaxCluster;
using attn::kMaxRep;
using attn::kMaxStages;

struct Scales {
  const float* k;
  const float* v;
};

// Largest decode CTA: one producer warp and a warp per KV head of the group.
constexpr int kMaxThreads = 9 * 32;

// Heads per CTA: the largest divisor of n_kv that is at most 8 (a row of 8
// heads is at most 1 KB).
inline int head_group(int n_kv) {
  int best = 1;
  for (int h = 1; h <= 8 && h <= n_kv; ++h)
    if (n_kv % h == 0) best = h;
  return best;
}

// attn::used_len and attn::check_length by ordinary loads: these kernels start
// while the lengths may still be written (see kv_fp8.cu's pdl_wait).
__device__ __forceinline__ int length_of(const DecodeParams& p, int b) {
  return max(0, min(p.seq_lens[b], p.max_len));
}

__device__ __forceinline__ void report_bad_length(const DecodeParams& p, int b) {
  const int L = p.seq_lens[b];
  if (L < 0 || L > p.max_seq_len) report(p.err, PKV_DEVERR_LENGTH);
  else if (L > p.W * kBS) report(p.err, PKV_DEVERR_TABLE_WIDTH);
}

// Lengths that a CTA which plans for itself keeps in shared memory (larger
// batches read them again where they are needed).
constexpr int kKeptLens = 1024;

// Walks a CTA's contiguous range of units segment by segment: a segment is the
// run of one (sequence, head group)'s blocks inside the range.
struct Walk {
  const DecodeParams& p;
  const int* lens;  // kept lengths, or null
  int b = 0, grp = 0, j = 0, L = 0, nblk = 1;

  __device__ __forceinline__ void enter() {
    L = lens != nullptr ? lens[b] : length_of(p, b);
    nblk = (L + kBS - 1) / kBS;
  }
  __device__ __forceinline__ void begin(int4 st) {
    b = st.x, grp = st.y, j = st.z;
    enter();
  }
  // past n units of the current group
  __device__ __forceinline__ void advance(int n) {
    j += n;
    if (j < nblk) return;
    j = 0;
    if (++grp < p.n_groups) return;
    grp = 0;
    do {
      if (++b >= p.B) {  // past the last unit: never used
        nblk = 1;
        return;
      }
      enter();
    } while (nblk == 0);
  }
};

// tc::tma_load_3d with an L2 cache policy for the copied lines.
__device__ __forceinline__ void tma_load_3d_hint(void* dst, const CUtensorMap* map, int x, int y,
                                                 int z, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar)),
      "l"(policy)
      : "memory");
}

// A place in the ring: its stage and how often the ring has been gone round
// (kept as counters: a division per block would cost as much as its copies).
struct RingPos {
  int st = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next(const Ring& r) {
    if (++st == r.nstages) {
      st = 0;
      ++round;
    }
  }
};

// Producer, one lane (elect_one): fetches blocks into the ring one after the
// other.  A block takes it about 200 cycles, and a stage of 8 heads x 64 dims
// should leave HBM every 700.
struct Producer {
  const Ring& ring;
  const CUtensorMap* tm_k;
  const CUtensorMap* tm_v;
  int num_blocks;
  int32_t* err;
  uint64_t policy;  // nonzero: an L2 cache policy for the copied lines
  RingPos pos;
  uint32_t issued = 0;

  // Block `id` (a bad one reads the zeros past the pool's end), from run
  // run0 of the tile map on (a run: `width` bytes of a row).  False on timeout.
  __device__ __forceinline__ bool fetch(int id, int run0) {
    const bool good = id >= 0 && id < num_blocks;
    if (!good) report(err, PKV_DEVERR_BLOCK_ID);
    if (pos.round > 0 && !wait_or_abort(ring.empty + pos.st, (pos.round - 1) & 1, ring.abort_flag)) {
      report(err, PKV_DEVERR_TIMEOUT);
      return false;
    }
    const int slot = (good ? id : num_blocks) * kBS;
    uint64_t* full = ring.full + pos.st;
    mbar_arrive_expect_tx(full, static_cast<uint32_t>(ring.stage_bytes));
    if (policy != 0) {
      tma_load_3d_hint(ring.k_tile(pos.st), tm_k, 0, slot, run0, full, policy);
      tma_load_3d_hint(ring.v_tile(pos.st), tm_v, 0, slot, run0, full, policy);
    } else {
      tc::tma_load_3d(ring.k_tile(pos.st), tm_k, 0, slot, run0, full);
      tc::tma_load_3d(ring.v_tile(pos.st), tm_v, 0, slot, run0, full);
    }
    pos.next(ring);
    ++issued;
    return true;
  }

  // Blocks row[0 .. n), ids read a group ahead.  False: gave up (and told the
  // consumers).
  __device__ __forceinline__ bool fetch_row(const int32_t* row, int n, int run0) {
    constexpr int kGroup = 8;
    int id[kGroup], next[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) next[i] = i < n ? row[i] : 0;
    for (int k0 = 0; k0 < n; k0 += kGroup) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i) id[i] = next[i];
#pragma unroll
      for (int i = 0; i < kGroup; ++i)
        next[i] = k0 + kGroup + i < n ? row[k0 + kGroup + i] : 0;
      if (*ring.abort_flag) return false;
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        if (k0 + i >= n) break;
        if (!fetch(id[i], run0)) {
          *ring.abort_flag = 1;
          return false;
        }
      }
    }
    return true;
  }

  // At the end: until the consumers have left the last tile, and all have landed;
  // where some thread gave up, a bounded wait for the copies still in flight, so
  // that none lands after the CTA has left.
  __device__ __forceinline__ void finish() const {
    if (issued == 0) return;
    const uint32_t last = issued - 1, st = last % ring.nstages;
    const bool left = wait_or_abort(ring.empty + st, (last / ring.nstages) & 1, ring.abort_flag);
    if (!left || *ring.abort_flag) attn::ring_drain(ring, issued);
  }
};

// Consumer warp: whether a thread of the CTA has given up (one of this warp for
// certain, since it set the flag).
__device__ __forceinline__ bool gave_up(const Ring& r) {
  return __any_sync(0xffffffffu, *r.abort_flag != 0);
}

__device__ __forceinline__ void release_tile(const Ring& r, const RingPos& pos) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(r.empty + pos.st);
}

// Tile map of an 8-bit pool: (width bytes, slot, run), read in boxes of one
// block's 16 slots x the runs of `heads` heads.
inline bool encode_tiles(CUtensorMap* map, const void* base, const PoolShape& pool, int width,
                         int heads) {
  const int row = pool.n_kv * pool.head_dim;
  const uint64_t dims[3] = {uint64_t(width), uint64_t(pool.num_blocks) * kBS, uint64_t(row / width)};
  const uint64_t strides[2] = {uint64_t(row), uint64_t(width)};
  const uint32_t box[3] = {uint32_t(width), kBS, uint32_t(heads * pool.head_dim / width)};
  return encode_u8(map, base, dims, strides, box, TileView::swizzle(width));
}

// A consumer warp's block scales, one block per lane.
struct ScaleBatch {
  float ks, vs, lv;
  // `id`: this lane's block (any value if it has none)
  __device__ __forceinline__ void load(const Scales& sc, const DecodeParams& p, int id, int head) {
    const bool ok = id >= 0 && id < p.num_blocks;  // others are read as zeros
    const int64_t at = int64_t(ok ? id : 0) * p.n_kv + head;
    ks = ok ? sc.k[at] : 1.f;
    vs = ok ? sc.v[at] : 1.f;
  }
  __device__ __forceinline__ void settle() { lv = __log2f(vs); }
};

// Consumer warp: its next NB tiles of the ring, blocks k .. k + NB - 1 of the
// batch in `sc`.  After a wait that gave up the warp goes on over what is there
// (its work is all its lanes'); gave_up tells before anything is stored.
template <int NB, typename RowsT>
__device__ __forceinline__ void take_tiles(RowsT& rows, const Ring& ring, RingPos& pos,
                                           const ScaleBatch& sc, int k, int j0, int valid,
                                           bool use, int32_t* err) {
  float ks[NB], vs[NB], lv[NB];
  const uint8_t *kt[NB], *vt[NB];
  RingPos at[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    ks[i] = __shfl_sync(0xffffffffu, sc.ks, (k + i) & 31);
    vs[i] = __shfl_sync(0xffffffffu, sc.vs, (k + i) & 31);
    lv[i] = __shfl_sync(0xffffffffu, sc.lv, (k + i) & 31);
    at[i] = pos;
    kt[i] = ring.k_tile(pos.st);
    vt[i] = ring.v_tile(pos.st);
    wait_or_flag(ring.full + pos.st, pos.round & 1, ring.abort_flag, err);
    pos.next(ring);
  }
  if (use) rows.template blocks<NB>(kt, vt, j0, valid, ks, vs, lv);
#pragma unroll
  for (int i = 0; i < NB; ++i) release_tile(ring, at[i]);
}

// CTAs of 8 consumer warps that an SM's registers hold.  A warp is a chain of
// latencies (tile, scores, maximum, weights, product), some 900 cycles a block
// whatever the head's width, and HBM brings a block of 8 x 64 in 720: narrow
// heads run on two CTAs an SM, with half the ring each, at 96 registers (bf16 at
// head_dim 64 spills 28 bytes there; more query rows or fp32's second terms at 64
// would spill much more).  One CTA -> two when it was chosen, 256 sequences of
// 2,048 tokens, 8 KV heads: head_dim 64 97.4 -> 88.2 us, 32 80.8 -> 56.8, 16 71.5 ->
// 49.2.
template <typename T, int HD, int NT>
constexpr int kCtasPerSm = NT == 1 && HD * int(sizeof(T)) / 2 <= 64 ? 2 : 1;

template <typename T, int HD, int NT, int CTAS>
__global__ void __launch_bounds__(kMaxThreads, CTAS)
    decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const DecodeParams p, const Scales sc, const int width) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int consumers = p.hg_size;
  Ring ring = attn::make_tile_ring(smem, p.nstages, kBS * p.hg_size * HD);
  attn::ring_init(ring, consumers);
  attn::pdl_wait();               // inputs and workspace belong to the preceding kernel
  attn::pdl_launch_dependents();  // the merge kernel may be scheduled (it waits for this grid)

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = gridDim.x;
  int U;
  int4 st = make_int4(0, 0, 0, 0);
  int* lens_s = reinterpret_cast<int*>(smem + p.part_off);  // [kKeptLens]
  const bool kept = p.plan_in_kernel && p.B <= kKeptLens;
  if (p.plan_in_kernel) {
    // scan the units per sequence in the (still unused) ring stages
    int* cu_s = reinterpret_cast<int*>(ring.stages);  // [B + 1]
    int* warp_tot = cu_s + p.B + 1;                   // [32]
    const int nt = blockDim.x;
    for (int b = threadIdx.x; b < p.B; b += nt) {
      if (blockIdx.x == 0) report_bad_length(p, b);
      const int L = length_of(p, b);
      if (kept) lens_s[b] = L;
      cu_s[b] = p.n_groups * ((L + kBS - 1) / kBS);
    }
    __syncthreads();
    const int chunk = (p.B + nt - 1) / nt;
    const int b0 = min(p.B, int(threadIdx.x) * chunk);
    const int b1 = min(p.B, b0 + chunk);
    int local = 0;
    for (int b = b0; b < b1; ++b) local += cu_s[b];
    int run = attn::cta_exclusive_scan(local, warp_tot);
    for (int b = b0; b < b1; ++b) {
      const int n = cu_s[b];
      cu_s[b] = run;
      run += n;
    }
    if (threadIdx.x == nt - 1) cu_s[p.B] = run;
    __syncthreads();
    U = cu_s[p.B];
    const int r0 = attn::range_begin(blockIdx.x, U, G);
    if (r0 < attn::range_begin(blockIdx.x + 1, U, G)) {
      const int b = attn::seq_of_unit(cu_s, p.B, r0);
      const int nblk = (cu_s[b + 1] - cu_s[b]) / p.n_groups;
      const int grp = (r0 - cu_s[b]) / nblk;
      st = make_int4(b, grp, (r0 - cu_s[b]) - grp * nblk, 0);
    }
    attn::zero_empty<T, HD>(p, blockIdx.x, G, [&](int b) { return cu_s[b + 1] == cu_s[b]; });
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      p.total_units[0] = U;
      p.total_units[1] = -1;  // a call planning for itself replaces any kept plan
    }
    fence_proxy_async_smem();  // the scan's stores come before the ring's copies
    __syncthreads();
  } else {
    U = __ldcg(p.total_units);
    st = __ldcg(p.starts + blockIdx.x);
  }
  const int r0 = attn::range_begin(blockIdx.x, U, G);
  const int r1 = attn::range_begin(blockIdx.x + 1, U, G);
  const int rows_per_group = p.hg_size * p.rep;
  Walk cur{p, kept ? lens_s : nullptr};
  if (r0 < r1) cur.begin(st);

  if (warp == consumers) {
    // -------------------------------------------------------- producer
    if (elect_one()) {
      const int nblk0 = cur.nblk;
      // (each block is read once: its lines leave L2 first)
      Producer pr{ring, &tm_k, &tm_v, p.num_blocks, p.err, tc::l2_evict_first_policy()};
      bool ok = true;
      for (int u = r0; u < r1 && ok;) {
        const int n = min(r1 - u, cur.nblk - cur.j);
        ok = pr.fetch_row(p.bt + int64_t(cur.b) * p.W + cur.j, n, cur.grp * p.hg_size * HD / width);
        u += n;
        cur.advance(n);
      }
      // the split group this CTA merges (read by the merge kernel)
      p.splits[blockIdx.x] =
          r0 < r1 ? attn::split_entry(blockIdx.x, G, U, st.x, st.y, st.z, nblk0)
                  : make_int4(-1, 0, 0, 0);
      pr.finish();
    }
  } else if (warp < consumers) {
    // ------------------------------------------------------- consumers
    Rows<T, HD, NT, false> rows;
    rows.place(width, warp);
    RingPos pos;
    const T* q = static_cast<const T*>(p.q);
    T* out = static_cast<T*>(p.out);
    for (int u = r0; u < r1;) {
      const int n = min(r1 - u, cur.nblk - cur.j);
      const int b = cur.b;
      const int kv_head = cur.grp * p.hg_size + warp;
      const int head0 = kv_head * p.rep;
      const int last = cur.L - 1;
      // block ids a batch of 32 ahead of the scales, scales a batch ahead of use
      const int32_t* row = p.bt + int64_t(b) * p.W + cur.j;
      auto id_at = [&](int i) { return i < n ? row[i] : -1; };
      ScaleBatch now, next;
      next.load(sc, p, id_at(lane), kv_head);
      int ids = id_at(32 + lane);
      rows.begin(
          [&](int r) -> const T* {
            return r < p.rep ? q + (int64_t(b) * p.n_heads + head0 + r) * HD : nullptr;
          },
          [&](int) { return last; }, p.scale_log2);
      constexpr int PAIR = Rows<T, HD, NT, false>::PAIR;
      for (int k = 0; k < n;) {
        if ((k & 31) == 0) {
          if (gave_up(ring)) break;
          now = next;
          now.settle();
          next.load(sc, p, ids, kv_head);
          ids = id_at(k + 64 + lane);
        }
        const int j0 = (cur.j + k) * kBS;
        if (PAIR == 2 && k + 1 < n) {
          take_tiles<PAIR>(rows, ring, pos, now, k, j0, cur.L - j0, true, p.err);
          k += PAIR;
        } else {
          take_tiles<1>(rows, ring, pos, now, k, j0, cur.L - j0, true, p.err);
          ++k;
        }
      }
      if (gave_up(ring)) break;
      if (cur.j == 0 && n == cur.nblk) {
        rows.store([&](int r) -> T* {
          return r < p.rep ? out + (int64_t(b) * p.n_heads + head0 + r) * HD : nullptr;
        });
      } else {  // a group split over several CTAs
        const int slot = 2 * blockIdx.x + (u == r0 ? 0 : 1);
        const int64_t base = int64_t(slot) * rows_per_group + warp * p.rep;
        rows.store_partial(
            [&](int r) -> float* { return r < p.rep ? p.ws_o + (base + r) * HD : nullptr; },
            [&](int r) -> float* { return p.ws_ml + (base + r) * 2; });
      }
      u += n;
      cur.advance(n);
    }
  }
}

// Batches too small to stream: one cluster of C CTAs per (sequence, head
// group), each a contiguous part of the sequence's at most 8 * C blocks, the
// parts combined through distributed shared memory (as the bf16 decode's
// cluster path; no workspace, no merge launch).
template <typename T, int HD, int NT>
__global__ void __launch_bounds__(kMaxThreads, 1)
    decode_cluster_kernel(const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const DecodeParams p,
                          const Scales sc, const int width) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int consumers = p.hg_size;
  Ring ring = attn::make_tile_ring(smem, p.nstages, kBS * p.hg_size * HD);
  attn::ring_init(ring, consumers);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = p.cluster;
  const int rank = static_cast<int>(cluster_ctarank());
  const int seg = static_cast<int>(blockIdx.x) / C;  // (sequence, head group)
  const int b = seg / p.n_groups;
  const int grp = seg - b * p.n_groups;
  const int rows_per_group = p.hg_size * p.rep;
  float* part_o = reinterpret_cast<float*>(smem + p.part_off);  // [rows_per_group][HD]
  float* part_ml = part_o + rows_per_group * HD;                // [rows_per_group][2]

  attn::pdl_wait();
  attn::pdl_launch_dependents();
  const int32_t* trow = p.bt + int64_t(b) * p.W;
  const int L = length_of(p, b);
  const int nblk = (L + kBS - 1) / kBS;
  const int j0 = rank * nblk / C, j1 = (rank + 1) * nblk / C;
  if (blockIdx.x == 0 && threadIdx.x == 0)
    p.total_units[1] = -1;  // a call planning for itself replaces any kept plan
  if (rank == 0 && grp == 0 && threadIdx.x == 0) report_bad_length(p, b);

  uint32_t issued = 0;
  if (warp == consumers) {
    if (elect_one()) {
      Producer pr{ring, &tm_k, &tm_v, p.num_blocks, p.err, tc::l2_evict_first_policy()};
      pr.fetch_row(trow + j0, j1 - j0, grp * p.hg_size * HD / width);
      issued = pr.issued;
    }
  } else if (warp < consumers) {
    const T* q = static_cast<const T*>(p.q);
    const int kv_head = grp * p.hg_size + warp;
    const int head0 = kv_head * p.rep;
    // scales of blocks j0 + lane (j1 - j0 <= 8)
    ScaleBatch now;
    now.load(sc, p, j0 + lane < j1 ? trow[j0 + lane] : -1, kv_head);
    Rows<T, HD, NT, false> rows;
    rows.place(width, warp);
    rows.begin(
        [&](int r) -> const T* {
          return r < p.rep ? q + (int64_t(b) * p.n_heads + head0 + r) * HD : nullptr;
        },
        [&](int) { return L - 1; }, p.scale_log2);
    now.settle();
    RingPos pos;
    constexpr int PAIR = Rows<T, HD, NT, false>::PAIR;
    for (int j = j0; j < j1;) {
      const int jp = j * kBS;
      if (PAIR == 2 && j + 1 < j1) {
        take_tiles<PAIR>(rows, ring, pos, now, j - j0, jp, L - jp, true, p.err);
        j += PAIR;
      } else {
        take_tiles<1>(rows, ring, pos, now, j - j0, jp, L - jp, true, p.err);
        ++j;
      }
    }
    // this CTA's part (also after an abort, so the barrier below is reached)
    rows.store_partial(
        [&](int r) -> float* { return r < p.rep ? part_o + (warp * p.rep + r) * HD : nullptr; },
        [&](int r) -> float* { return part_ml + (warp * p.rep + r) * 2; });
  }

  cluster_sync();  // every CTA's partial is in its shared memory
  if (*ring.abort_flag) attn::ring_drain(ring, issued);  // (as Producer::finish)
  // CTA `rank` combines elements [rank E / C, (rank + 1) E / C) of the group
  const int E = rows_per_group * HD;
  const int e0 = rank * E / C, e1 = (rank + 1) * E / C;
  T* out = static_cast<T*>(p.out) + (int64_t(b) * p.n_heads + int64_t(grp) * rows_per_group) * HD;
  for (int e = e0 + static_cast<int>(threadIdx.x); e < e1; e += static_cast<int>(blockDim.x)) {
    const int r = e / HD;
    float2 ml[kMaxCluster];
    float oc[kMaxCluster];
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {  // every peer's values in one round trip
      ml[c] = make_float2(-INFINITY, 0.f);
      oc[c] = 0.f;
      if (c < C) {
        ml[c] = ld_cluster_f32x2(cluster_map(part_ml + r * 2, c));
        oc[c] = ld_cluster_f32(cluster_map(part_o + e, c));
      }
    }
    float M = -INFINITY;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c)
      if (ml[c].y > 0.f) M = fmaxf(M, ml[c].x);  // a part that saw no key has no weight
    float acc = 0.f, den = 0.f;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
      if (ml[c].y > 0.f) {
        const float w = fast_exp2(ml[c].x - M) * ml[c].y;
        den += w;
        acc = fmaf(w, oc[c], acc);
      }
    }
    out[e] = Elem<T>::from_f(den > 0.f ? acc * (1.f / den) : 0.f);
  }
  cluster_sync();  // the peers have read this CTA's partials
}

// Joins the split group that CTA x of the decode merges: its parts' outputs
// weighted by 2^(M - max M) l, one float4 of the group's rows a thread.  As the
// bf16 decode's merge, but a group's rows lie over several small CTAs (y), which
// fit an SM beside a decode's CTA (this call's, and the next one's, which is
// there early): 64 sequences of 512 - 2,048 tokens of 8 x 128, 32 heads, take
// 33.4 us in place of 35.4, of 8 x 64 24.1 in place of 24.9.
constexpr int kJoinThreads = 128;

template <typename T, int HD>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const DecodeParams p) {
  constexpr int NB = 4;  // parts in flight
  attn::pdl_launch_dependents();
  attn::pdl_wait();  // the decode's partials and split entries
  const int4 sp = __ldcg(p.splits + blockIdx.x);
  if (sp.x < 0) return;
  const int rows = p.hg_size * p.rep;
  const int E = rows * HD;  // elements of a part
  const int e = (blockIdx.y * blockDim.x + threadIdx.x) * 4;
  if (e >= E) return;
  const bool c0_tail = (sp.y & attn::kSplitC0Tail) != 0;
  const bool dense = (sp.y & attn::kSplitDense) != 0;
  const int U = dense ? 0 : __ldcg(p.total_units);  // only sparse grids look at range starts
  const int G = p.grid;
  const int c0 = sp.z & 0xffff, c1 = static_cast<int>(static_cast<uint32_t>(sp.z) >> 16);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, den = 0.f;
  for (int cs = c0; cs <= c1; cs += NB) {
    float4 o[NB];
    float2 ml[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int c = cs + k;
      o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      ml[k] = make_float2(-INFINITY, 0.f);
      if (c <= c1 && (dense || attn::range_begin(c + 1, U, G) > attn::range_begin(c, U, G))) {
        // c0 holds the group's first units at the end of its range, unless its
        // range starts at the group
        const int64_t slot = 2 * c + (c == c0 && c0_tail ? 1 : 0);
        o[k] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + slot * E + e));
        ml[k] = __ldcg(reinterpret_cast<const float2*>(p.ws_ml + (slot * rows + e / HD) * 2));
      }
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      if (ml[k].y > 0.f) {  // a part that saw no key has no weight
        const float Mn = fmaxf(M, ml[k].x);
        const float a = fast_exp2(M - Mn);
        const float w = fast_exp2(ml[k].x - Mn) * ml[k].y;
        acc = make_float4(fmaf(w, o[k].x, acc.x * a), fmaf(w, o[k].y, acc.y * a),
                          fmaf(w, o[k].z, acc.z * a), fmaf(w, o[k].w, acc.w * a));
        den = fmaf(den, a, w);
        M = Mn;
      }
    }
  }
  const int64_t row0 = int64_t(sp.x) * p.n_heads + (sp.y & 0xffff) * rows;
  T* out = static_cast<T*>(p.out) + row0 * HD + e;
  const float inv = den > 0.f ? 1.f / den : 0.f;
  const float4 v = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(out) = v;
  } else {
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
}

// --------------------------------------------------------------- host side

template <typename T, int HD, int NT>
struct DecodeFp8 {
  static constexpr int kSmemMax = 226 * 1024;  // what both kernels opt in to
  static int stage_bytes(int hg) { return 2 * kBS * hg * HD; }
  // barriers, alignment slack and ring; what follows starts there
  static size_t smem_for(int hg, int nstages) {
    return kBarrierBytes + 1024 + size_t(nstages) * stage_bytes(hg);
  }
  // 2: CTAs for twice 8 consumer warps an SM.  Not for groups whose rows are not
  // whole 128 bytes, whose copies are twice as many: 256 sequences of 2,048
  // tokens, 9 heads on 3 of 64, take 52.4 us so and 49.3 with one CTA's registers.
  static int doubled(int hg) { return tile_width(hg, HD) == 128 ? kCtasPerSm<T, HD, NT> : 1; }
  static auto kernel(int hg) {
    return doubled(hg) == 2 ? decode_kernel<T, HD, NT, kCtasPerSm<T, HD, NT>>
                            : decode_kernel<T, HD, NT, 1>;
  }
  // Ring depth: about 176 KB of stages per SM, shared by the CTAs of 8
  // consumer warps in all (narrow groups: several CTAs per SM, each with its
  // barriers and kept lengths).
  static int ring_stages(int hg) {
    const int ctas = std::max(1, 8 / hg) * doubled(hg);
    const int ns = (176 - 4 * (ctas - 1)) * 1024 / ctas / stage_bytes(hg);
    return std::max(2, std::min(kMaxStages, ns));
  }
  static cudaError_t grid(const AttnArgs& a, int hg, int* G, size_t* smem, int* nstages, int* wave) {
    *nstages = ring_stages(hg);
    *smem = smem_for(hg, *nstages) + kKeptLens * 4;
    static KernelSetup setup[2];
    int per_sm = 0;
    const cudaError_t e = kernel_setup(setup[doubled(hg) - 1], kernel(hg), static_cast<int>(*smem),
                                       (hg + 1) * 32, &per_sm, kSmemMax);
    if (e != cudaSuccess) return e;
    per_sm = std::max(1, std::min(per_sm, 16));  // 16: what the workspace is sized for
    *G = sm_count() * per_sm;
    *wave = *G / doubled(hg);
    if (a.max_ctas > 0 && a.max_ctas < *G) *G = a.max_ctas;
    const int64_t max_units = int64_t(a.num_seqs) * (a.pool.n_kv / hg) *
                              ((int64_t(a.max_seq_len) + kBS - 1) / kBS);
    if (max_units < *G) *G = static_cast<int>(std::max<int64_t>(1, max_units));
    return cudaSuccess;
  }

  static cudaError_t run(const AttnArgs& a, const Scales& sc, cudaStream_t stream) {
    const PoolShape& pool = a.pool;
    const int hg = head_group(pool.n_kv);
    DecodeParams p{};
    p.q = a.q;
    p.out = a.out;
    p.k_pool = static_cast<const uint8_t*>(a.k_pool);
    p.v_pool = static_cast<const uint8_t*>(a.v_pool);
    p.bt = a.block_tables;
    p.seq_lens = a.seq_lens;
    p.err = a.err;
    p.B = a.num_seqs;
    p.n_heads = a.n_heads;
    p.n_kv = pool.n_kv;
    p.rep = a.n_heads / pool.n_kv;
    p.hg_size = hg;
    p.n_groups = pool.n_kv / hg;
    p.W = a.max_blocks_per_seq;
    p.num_blocks = pool.num_blocks;
    p.max_len = a.max_seq_len;  // (no more than the tables hold)
    p.max_seq_len = a.max_seq_len;
    p.head_dim = HD;
    p.elem_bytes = 1;
    p.scale_log2 = a.scale * attn::kLog2e;
    int G = 0, wave = 0;
    size_t smem = 0;
    cudaError_t e = grid(a, hg, &G, &smem, &p.nstages, &wave);
    if (e != cudaSuccess) return e;
    if (G > 65535) return cudaErrorInvalidValue;  // split entries pack CTA indices in 16 bits
    p.grid = G;
    const DecodeWs L(a.num_seqs, G, size_t(hg) * p.rep, HD);
    if (L.total > a.workspace_bytes) return cudaErrorInvalidValue;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    p.cu_units = reinterpret_cast<int32_t*>(ws + L.cu);
    p.starts = reinterpret_cast<int4*>(ws + L.starts);
    p.splits = reinterpret_cast<int4*>(ws + L.splits);
    p.total_units = reinterpret_cast<int32_t*>(ws + L.total_units);
    p.ws_ml = reinterpret_cast<float*>(ws + L.ml);
    p.ws_o = reinterpret_cast<float*>(ws + L.o);
    CUtensorMap tm_k{}, tm_v{};
    const int width = tile_width(hg, HD);
    if (!encode_tiles(&tm_k, a.k_pool, pool, width, hg) ||
        !encode_tiles(&tm_v, a.v_pool, pool, width, hg))
      return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3((hg + 1) * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;

    // Latency-bound batches, by the rule of the bf16 decode: the longest
    // sequence at most 64 blocks and the clusters within two waves.
    const int nmax = p.max_len / kBS + (p.max_len % kBS != 0);
    const int C = std::max(1, std::min(kMaxCluster, (nmax + 3) / 4));
    const int64_t ctas = int64_t(p.B) * p.n_groups * C;
    if (a.max_ctas == 0 && nmax <= 8 * kMaxCluster && ctas <= 2 * int64_t(wave)) {
      p.cluster = C;
      p.nstages = std::max(2, std::min(p.nstages, (nmax + C - 1) / C));
      const size_t rows = size_t(hg) * p.rep;
      const size_t extra = rows * HD * 4 + (rows * 2 * 4 + 15) / 16 * 16;
      while (p.nstages > 2 && smem_for(hg, p.nstages) + extra > size_t(kSmemMax)) --p.nstages;
      p.part_off = static_cast<int>(smem_for(hg, p.nstages));
      static KernelSetup setup;
      e = kernel_setup(setup, decode_cluster_kernel<T, HD, NT>, kSmemMax, (hg + 1) * 32,
                       nullptr);
      if (e != cudaSuccess) return e;
      attr[1].id = cudaLaunchAttributeClusterDimension;
      attr[1].val.clusterDim.x = static_cast<unsigned>(C);
      attr[1].val.clusterDim.y = 1;
      attr[1].val.clusterDim.z = 1;
      cfg.numAttrs = 2;
      cfg.gridDim = dim3(static_cast<unsigned>(ctas));
      cfg.dynamicSmemBytes = p.part_off + extra;
      e = cudaLaunchKernelEx(&cfg, decode_cluster_kernel<T, HD, NT>, tm_k, tm_v, p, sc, width);
      return e != cudaSuccess ? e : cudaGetLastError();
    }
    p.part_off = static_cast<int>(smem_for(hg, p.nstages));  // the kept lengths
    // every CTA scans the lengths in its ring stages; larger batches have a
    // plan kernel
    p.plan_in_kernel = a.num_seqs <= kKernelPlanSeqs &&
                       size_t(a.num_seqs + 1 + 32) * 4 <= size_t(p.nstages) * stage_bytes(hg);
    if (!p.plan_in_kernel) {
      attn::decode_plan_kernel<T, HD><<<1, 1024, 0, stream>>>(p);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    cfg.gridDim = dim3(G);
    cfg.dynamicSmemBytes = smem;
    e = cudaLaunchKernelEx(&cfg, kernel(hg), tm_k, tm_v, p, sc, width);
    if (e != cudaSuccess) return e;
    const int vecs = hg * p.rep * HD / 4;  // of a group's rows
    const int threads = std::min(kJoinThreads, (vecs + 31) / 32 * 32);
    cfg.gridDim = dim3(G, (vecs + threads - 1) / threads);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, join_kernel<T, HD>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
};

template <typename T>
cudaError_t decode_as(const AttnArgs& a, const Scales& sc, cudaStream_t s) {
  const bool one = a.n_heads / a.pool.n_kv <= 8;
  switch (a.pool.head_dim) {
    case 16: return one ? DecodeFp8<T, 16, 1>::run(a, sc, s) : DecodeFp8<T, 16, 2>::run(a, sc, s);
    case 32: return one ? DecodeFp8<T, 32, 1>::run(a, sc, s) : DecodeFp8<T, 32, 2>::run(a, sc, s);
    case 64: return one ? DecodeFp8<T, 64, 1>::run(a, sc, s) : DecodeFp8<T, 64, 2>::run(a, sc, s);
    default: return one ? DecodeFp8<T, 128, 1>::run(a, sc, s) : DecodeFp8<T, 128, 2>::run(a, sc, s);
  }
}

// The two output types are compiled in their own translation units.
cudaError_t decode_fp8_bf16(const AttnArgs& a, const Scales& sc, cudaStream_t s);
cudaError_t decode_fp8_f32(const AttnArgs& a, const Scales& sc, cudaStream_t s);

}  // namespace fp8
}  // namespace pkv
