// Decode over the 4-bit cache: one query per sequence attends to the sequence's pages
// (mathematics and layouts of the tiles in fp4_rows.cuh).
//
// Bound by reading the cache, 9 / 8 x n_kv x head_dim bytes a token, and close behind by
// the instructions that turn codes into f16 operands: 292 a block and head of 128 (187 of
// 64), where the SM's schedulers have 397 in the time that the block takes to arrive.  So
// nothing is spent on synchronisation: a head's rows of a block lie together in the
// pools (four runs: K and V, codes and scales, 2.3 KB at head_dim 128), and each warp
// fetches its own into a ring of its own, by asynchronous 16-byte copies of all its lanes
// as soon as it has left a stage.  No warp waits for another, and there is no barrier.
// (Bulk copies would be issued one by one, some 25 instructions each: 142 us for 256
// sequences of 16 - 8,192 tokens, 64 heads on 8 of 128, which take 108 so.)
//
// Work split: one CTA or one thread-block cluster per (sequence, head group), combined
// through distributed shared memory, where that fills the GPU evenly enough; else equal
// contiguous ranges of (sequence, head group, block) units, one per CTA of a persistent
// grid, and a joining kernel for the groups that several CTAs share.  Either way a warp for
// each KV head of the group, so that the heads of a block, which lie together, are read at
// about the same time (ranges of (sequence, head, block) units for each warp by itself: 117
// us for those 256 sequences, 94 for the copies alone; these 111 and 90).
//
// Those 256 sequences: 108 us, 5.0 TB/s, of which the joining launch takes 6.3 and the
// partial results 2.5; issue slots are 63% taken, the ALUs 54%.  64 sequences of 512 - 2,048
// tokens, 32 heads on 8 of 64: 22.5 us in clusters of four.
#pragma once

#include <algorithm>
#include <type_traits>

#include "attention.cuh"
#include "decode_fp8.cuh"
#include "fp4_rows.cuh"

namespace pkv {
namespace fp4 {

using attn::DecodeParams;
using attn::DecodeWs;
using attn::kKernelPlanSeqs;
using attn::kMaxCluster;
using fp8::Walk;
using fp8::head_group;
using fp8::kKeptLens;
using fp8::length_of;
using fp8::report_bad_length;

constexpr int kWarps = 8;       // of a CTA at the most: a head group's
constexpr int kMaxBlocks = 32;  // of a warp of a cluster: a warp's lanes hold their ids
constexpr int kMaxStages = 12;  // of a warp's ring
constexpr int kSmemMax = 226 * 1024;  // of an SM's CTAs

// The pools as they are read.
struct Pools {
  const uint8_t *k, *v, *kg, *vg;
  const float *k_scale, *v_scale;
  explicit Pools(const Fp4Cache& c)
      : k(static_cast<const uint8_t*>(c.k_pool)),
        v(static_cast<const uint8_t*>(c.v_pool)),
        kg(static_cast<const uint8_t*>(c.k_groups)),
        vg(static_cast<const uint8_t*>(c.v_groups)),
        k_scale(c.k_scale),
        v_scale(c.v_scale) {}
};

// 16 bytes global -> shared past L1, with an L2 cache policy; zeros where size is 0.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, uint32_t size,
                                       uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
               "r"(size), "l"(policy)
               : "memory");
}

__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Until at most N of this lane's groups of copies are on their way; then, for the warp, the
// groups before those are there.
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
  __syncwarp();
}

// Fetches one head's blocks, by a whole warp: a lane copies 16-byte pieces of the four runs.
template <int HD>
struct Fetcher {
  static constexpr bool kWide = HD >= 64;  // K's codes are a warp's copies or more
  const uint8_t *codes, *codes_v, *groups;  // this lane's first pieces, in head 0 of block 0
  uint32_t at_codes, at_groups;             // and in a tile
  bool has_codes, has_groups;
  int n_kv, num_blocks;
  int32_t* err;
  uint64_t policy;

  __device__ __forceinline__ Fetcher(const Pools& pools, int n_kv_, int num_blocks_, int32_t* err_)
      : n_kv(n_kv_), num_blocks(num_blocks_), err(err_), policy(tc::l2_evict_first_policy()) {
    using TileT = Tile<HD>;
    const int lane = threadIdx.x & 31;
    // codes: K's pieces, then V's (wide heads: both in every lane)
    constexpr int nc = TileT::kCodes / 16, ng = TileT::kGroups / 16;
    const bool v = !kWide && lane >= nc;
    const int piece = kWide ? lane : v ? lane - nc : lane;
    has_codes = kWide || lane < 2 * nc;
    codes = (v ? pools.v : pools.k) + piece * 16;
    codes_v = pools.v + piece * 16;
    at_codes = (v ? TileT::kVCodes : 0) + piece * 16;
    // scales: in the lanes that follow (narrowest heads) or in a round of their own
    const int g = HD == 16 ? lane - 2 * nc : lane;
    has_groups = g >= 0 && g < 2 * ng;
    groups = g < ng ? pools.kg + g * 16 : pools.vg + (g - ng) * 16;
    at_groups = TileT::kKGroups + g * 16;
  }
  // Head `head` of block `id` (every lane's the same) into the tile at shared address
  // `tile`; a bad id reads zeros.
  __device__ __forceinline__ void block(uint32_t tile, int id, int head) const {
    using TileT = Tile<HD>;
    uint32_t size = 16u;
    if (static_cast<uint32_t>(id) >= static_cast<uint32_t>(num_blocks)) {
      if ((threadIdx.x & 31) == 0) report(err, PKV_DEVERR_BLOCK_ID);
      size = 0u;
      id = 0;
    }
    const uint32_t row = static_cast<uint32_t>(id) * n_kv + head;  // (below 2^31)
    const uint8_t* k = codes + uint64_t(row) * TileT::kCodes;
    if constexpr (kWide) {
      const uint8_t* v = codes_v + uint64_t(row) * TileT::kCodes;
#pragma unroll
      for (int i = 0; i < TileT::kCodes / 512; ++i) {
        copy16(tile + at_codes + i * 512, k + i * 512, size, policy);
        copy16(tile + at_codes + TileT::kVCodes + i * 512, v + i * 512, size, policy);
      }
    } else if (has_codes) {
      copy16(tile + at_codes, k, size, policy);
    }
    if (has_groups) copy16(tile + at_groups, groups + uint64_t(row) * TileT::kGroups, size, policy);
  }
};

// The CTA whose range holds unit u of U, of G CTAs: the largest c with floor(c U / G) <= u.
__device__ __forceinline__ int owner_of(int u, int U, int G) {
  const uint64_t n = uint64_t(uint32_t(u) + 1u) * uint32_t(G) - 1u;
  if (n <= 0xffffffffull) return static_cast<int>(uint32_t(n) / uint32_t(U));  // (far shorter)
  return static_cast<int>(n / uint32_t(U));
}

// The split entry of CTA c (of G, over U units) whose range starts at block j of a group
// of nblk blocks: attn::split_entry, its owners by division.
__device__ __forceinline__ int4 split_entry(int c, int G, int U, int b, int grp, int j, int nblk) {
  if (j == 0) return make_int4(-1, 0, 0, 0);
  const int first = attn::range_begin(c, U, G) - j;  // the group's first unit
  const int c0 = owner_of(first, U, G);
  // (the second of its CTAs joins them)
  if (owner_of(attn::range_begin(c0 + 1, U, G), U, G) != c) return make_int4(-1, 0, 0, 0);
  const int flags = (attn::range_begin(c0, U, G) != first ? attn::kSplitC0Tail : 0) |
                    (U >= G ? attn::kSplitDense : 0);
  return make_int4(b, grp | flags, c0 | (owner_of(first + nblk - 1, U, G) << 16), first);
}

// Units before each sequence, by a converged warp: for batches of at most 32 kLaneSeqs
// sequences a scan in registers, without a barrier.
constexpr int kLaneSeqs = 8;

struct WarpScan {
  int n[kLaneSeqs];  // units of sequences first .. first + per - 1
  int first, per, before, total;

  __device__ __forceinline__ explicit WarpScan(const DecodeParams& p) {
    const int lane = threadIdx.x & 31;
    per = (p.B + 31) / 32;
    first = lane * per;
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kLaneSeqs; ++i) {
      n[i] = 0;
      if (i < per && first + i < p.B) n[i] = p.n_groups * ((length_of(p, first + i) + kBS - 1) / kBS);
    }
#pragma unroll
    for (int i = 0; i < kLaneSeqs; ++i) sum += n[i];
    before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    total = __shfl_sync(0xffffffffu, before, 31);
    before -= sum;
  }
  // The sequence that holds unit u < total: its number, its first unit and its units.
  __device__ __forceinline__ int3 find(int u) const {
    int3 r = make_int3(-1, 0, 0);
    int at = before;
#pragma unroll
    for (int i = 0; i < kLaneSeqs; ++i) {
      if (u >= at && u < at + n[i]) r = make_int3(first + i, at, n[i]);
      at += n[i];
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, r.x >= 0)) - 1;
    return make_int3(__shfl_sync(0xffffffffu, r.x, src), __shfl_sync(0xffffffffu, r.y, src),
                     __shfl_sync(0xffffffffu, r.z, src));
  }
  // Sequence b's first unit and units.
  __device__ __forceinline__ int2 of(int b) const {
    const int src = b / per, k = b - src * per;
    int at = before, units = 0;
#pragma unroll
    for (int i = 0; i < kLaneSeqs; ++i) {
      if (i < k) at += n[i];
      if (i == k) units = n[i];
    }
    return make_int2(__shfl_sync(0xffffffffu, at, src), __shfl_sync(0xffffffffu, units, src));
  }
};

// CTAs of eight warps that an SM's registers hold (or as many more narrower ones).
template <typename T, int HD, int NT>
constexpr int kCtasPerSm = NT == 1 && HD * int(sizeof(T)) / 2 <= 128 ? 2 : 1;

// A ring's depth, as the SM's shared memory allows (with the kept lengths).
template <typename T, int HD, int NT>
constexpr int kStages = std::min(kMaxStages,
                                 (kSmemMax / kCtasPerSm<T, HD, NT> - kKeptLens * 4 - 1024) /
                                     (kWarps * Tile<HD>::kBytes));

template <typename T, int HD, int NT>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm<T, HD, NT>)
    decode_kernel(const DecodeParams p, const Pools pools) {
  extern __shared__ __align__(128) uint8_t smem[];  // [kWarps][kStages] tiles, kept lengths
  constexpr int S = kStages<T, HD, NT>;
  attn::pdl_wait();               // inputs and workspace belong to the preceding kernel
  attn::pdl_launch_dependents();  // the joining kernel may be scheduled (it waits for this grid)

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = gridDim.x;
  const int me = blockIdx.x;
  int U, r0, r1;  // all units, this CTA's range of them
  int4 st = make_int4(0, 0, 0, 0);
  int* lens_s = reinterpret_cast<int*>(smem + p.part_off);  // [kKeptLens]
  const bool kept = p.plan_in_kernel && p.part_off != 0 && p.B <= kKeptLens;
  if (p.B <= 32 * kLaneSeqs) {
    // (one warp finds the CTA's place for all: 0.2 - 0.3 us less than each for itself)
    __shared__ int4 range_s, start_s;
    if (warp == 0) {
      const WarpScan scan(p);
      U = scan.total;
      r0 = attn::range_begin(me, U, G);
      r1 = attn::range_begin(me + 1, U, G);
      if (r0 < r1) {
        const int3 seq = scan.find(r0);
        const int nblk = seq.z / p.n_groups;
        const int grp = (r0 - seq.y) / nblk;
        st = make_int4(seq.x, grp, (r0 - seq.y) - grp * nblk, 0);
      }
      if (lane == 0) {
        range_s = make_int4(r0, r1, U, 0);
        start_s = st;
        if (me == 0) {
          p.total_units[0] = U;
          p.total_units[1] = -1;  // a call planning for itself replaces any kept plan
        }
      }
    }
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
      if (kept) lens_s[b] = length_of(p, b);
      if (blockIdx.x == 0) report_bad_length(p, b);
    }
    attn::zero_empty<T, HD>(p, blockIdx.x, G, [&](int b) { return length_of(p, b) == 0; });
    __syncthreads();
    r0 = range_s.x, r1 = range_s.y, U = range_s.z;
    st = start_s;
  } else if (p.plan_in_kernel) {
    // scan the units per sequence in the (still unused) stages
    int* cu_s = reinterpret_cast<int*>(smem);  // [B + 1]
    int* warp_tot = cu_s + p.B + 1;            // [32]
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
    r0 = attn::range_begin(me, U, G);
    r1 = attn::range_begin(me + 1, U, G);
    if (r0 < r1) {
      const int b = attn::seq_of_unit(cu_s, p.B, r0);
      const int nblk = (cu_s[b + 1] - cu_s[b]) / p.n_groups;
      const int grp = (r0 - cu_s[b]) / nblk;
      st = make_int4(b, grp, (r0 - cu_s[b]) - grp * nblk, 0);
    }
    attn::zero_empty<T, HD>(p, blockIdx.x, gridDim.x, [&](int b) { return cu_s[b + 1] == cu_s[b]; });
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      p.total_units[0] = U;
      p.total_units[1] = -1;  // a call planning for itself replaces any kept plan
    }
    __syncthreads();  // (the stages are the rings' from here on)
  } else {
    U = __ldcg(p.total_units);
    r0 = attn::range_begin(me, U, G);
    r1 = attn::range_begin(me + 1, U, G);
    st = __ldcg(p.starts + me);
  }
  const int rows_per_group = p.hg_size * p.rep;
  if (r0 >= r1) {
    if (threadIdx.x == 0) p.splits[me] = make_int4(-1, 0, 0, 0);
    return;
  }
  uint8_t* ring = smem + warp * S * Tile<HD>::kBytes;
  const uint32_t ring_at = smem_addr(ring);
  const Fetcher<HD> fetch(pools, p.n_kv, p.num_blocks, p.err);
  Walk cur{p, kept ? lens_s : nullptr};
  cur.begin(st);

  // ---- the blocks on their way: a walk of its own, some stages ahead.  Lane i holds the
  // id of block fj + i of the walk's segment (its next 32).
  Walk ahead = cur;
  int left = r1 - r0, seg = min(left, ahead.nblk - ahead.j), k = 0, ids = 0;
  uint32_t fill = 0;  // offset of the next stage to fill
  auto feed = [&]() {
    if (left > 0) {
      if ((k & 31) == 0) {
        const int i = k + lane;
        if (i < seg) ids = p.bt[int64_t(ahead.b) * p.W + ahead.j + i];
      }
      fetch.block(ring_at + fill, __shfl_sync(0xffffffffu, ids, k & 31),
                  ahead.grp * p.hg_size + warp);
      fill = fill == (S - 1) * Tile<HD>::kBytes ? 0 : fill + Tile<HD>::kBytes;
      --left;
      if (++k == seg) {
        ahead.advance(seg);
        seg = min(left, ahead.nblk - ahead.j);
        k = 0;
      }
    }
    commit_copies();  // (an empty group past the last block: waits count groups)
  };
  // NB of them, of which most calls find all inside the segment and its 32 ids
  auto feed_some = [&](auto nb) {
    constexpr int NB = decltype(nb)::value;
    if (NB > 1 && (k & 31) != 0 && (k & 31) + NB <= 32 && k + NB < seg) {
      const int head = ahead.grp * p.hg_size + warp;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        fetch.block(ring_at + fill, __shfl_sync(0xffffffffu, ids, (k & 31) + i), head);
        fill = fill == (S - 1) * Tile<HD>::kBytes ? 0 : fill + Tile<HD>::kBytes;
        commit_copies();
      }
      left -= NB;
      k += NB;
    } else {
#pragma unroll 1
      for (int i = 0; i < NB; ++i) feed();
    }
  };
#pragma unroll 1
  for (int i = 0; i < S; ++i) feed();
  // (while the first blocks come)
  if (warp == 0) {
    const int4 entry = split_entry(me, G, U, st.x, st.y, st.z, cur.nblk);
    if (lane == 0) p.splits[me] = entry;
  }

  using RowsT = Rows<T, HD, NT, false>;
  RowsT rows;
  rows.place();
  uint32_t at = 0;  // offset of the stage of the next block
  // The warp's next NB tiles; their stages are filled again.  EDGE: some token may lie
  // past the sequence's end.
  auto take = [&](auto nb, auto edge, int j0) {
    constexpr int NB = decltype(nb)::value;
    const uint8_t* t[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      t[i] = ring + at;
      at = at == (S - 1) * Tile<HD>::kBytes ? 0 : at + Tile<HD>::kBytes;
    }
    wait_copies<S - NB>();
    rows.template blocks<NB, decltype(edge)::value>(t, j0, cur.L - j0);
    __syncwarp();
    feed_some(nb);
  };
  const T* q = static_cast<const T*>(p.q);
  T* out = static_cast<T*>(p.out);
  for (int u = r0; u < r1;) {
    const int n = min(r1 - u, cur.nblk - cur.j);
    const int kv_head = cur.grp * p.hg_size + warp;
    const int64_t row0 = int64_t(cur.b) * p.n_heads + int64_t(kv_head) * p.rep;
    const int last = cur.L - 1;
    rows.begin([&](int r) -> const T* { return r < p.rep ? q + (row0 + r) * HD : nullptr; },
               [&](int) { return last; }, p.scale_log2 * pools.k_scale[kv_head],
               pools.v_scale[kv_head]);
    const int full = min(n, cur.L / kBS - cur.j);  // blocks without an edge
    int i = 0;
    for (; i + RowsT::TAKE <= full; i += RowsT::TAKE)
      take(std::integral_constant<int, RowsT::TAKE>{}, std::false_type{}, (cur.j + i) * kBS);
    if (RowsT::TAKE > 2 && i + 2 <= full) {
      take(std::integral_constant<int, 2>{}, std::false_type{}, (cur.j + i) * kBS);
      i += 2;
    }
    for (; i < n; ++i) take(std::integral_constant<int, 1>{}, std::true_type{}, (cur.j + i) * kBS);
    if (cur.j == 0 && n == cur.nblk) {
      rows.store([&](int r) -> T* { return r < p.rep ? out + (row0 + r) * HD : nullptr; });
    } else {  // a group that several CTAs share
      const int64_t base = int64_t(2 * me + (u == r0 ? 0 : 1)) * rows_per_group + warp * p.rep;
      rows.store_partial(
          [&](int r) -> float* { return r < p.rep ? p.ws_o + (base + r) * HD : nullptr; },
          [&](int r) -> float* { return p.ws_ml + (base + r) * 2; });
    }
    u += n;
    cur.advance(n);
  }
}

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// One cluster of C CTAs per (sequence, head group), a warp per head of the group, each CTA
// a contiguous part of the sequence's at most kMaxBlocks * C blocks, the parts combined
// through distributed shared memory: no lengths to scan, no workspace, no joining launch.
template <typename T, int HD, int NT>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm<T, HD, NT>)
    decode_cluster_kernel(const DecodeParams p, const Pools pools) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int S = kStages<T, HD, NT>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = p.cluster;
  const int rank = static_cast<int>(cluster_ctarank());
  const int seg = static_cast<int>(blockIdx.x) / C;  // (sequence, head group)
  const int b = seg / p.n_groups;
  const int grp = seg - b * p.n_groups;
  const int rows_per_group = p.hg_size * p.rep;
  // a warp's ring, afterwards its part [rep][HD]; behind the rings the parts' references
  // and sums [rows_per_group][2]
  const int room = p.nstages;  // bytes
  uint8_t* ring = smem + warp * room;
  float* part_o = reinterpret_cast<float*>(ring);
  float* part_ml = reinterpret_cast<float*>(smem + p.part_off);

  attn::pdl_wait();
  attn::pdl_launch_dependents();
  const int L = length_of(p, b);
  const int nblk = (L + kBS - 1) / kBS;
  const int j0 = rank * nblk / C, n = (rank + 1) * nblk / C - j0;  // n <= kMaxBlocks
  if (blockIdx.x == 0 && threadIdx.x == 0)
    p.total_units[1] = -1;  // a call planning for itself replaces any kept plan
  if (rank == 0 && grp == 0 && threadIdx.x == 0) report_bad_length(p, b);
  const int kv_head = grp * p.hg_size + warp;
  const Fetcher<HD> fetch(pools, p.n_kv, p.num_blocks, p.err);
  const int ids = lane < n ? p.bt[int64_t(b) * p.W + j0 + lane] : 0;
  const uint32_t ring_at = smem_addr(ring);
  uint32_t fill = 0;  // offset of the next stage to fill (a ring with room for all is never full)
  int fed = 0;
  auto feed = [&]() {
    if (fed < n) {
      fetch.block(ring_at + fill, __shfl_sync(0xffffffffu, ids, fed), kv_head);
      fill = fill == (S - 1) * Tile<HD>::kBytes ? 0 : fill + Tile<HD>::kBytes;
      ++fed;
    }
    commit_copies();  // (an empty group past the last block: waits count groups)
  };
#pragma unroll 1
  for (int i = 0; i < S; ++i) feed();
  using RowsT = Rows<T, HD, NT, false>;
  const T* q = static_cast<const T*>(p.q) + (int64_t(b) * p.n_heads + int64_t(kv_head) * p.rep) * HD;
  RowsT rows;
  rows.place();
  rows.begin([&](int r) -> const T* { return r < p.rep ? q + r * HD : nullptr; },
             [&](int) { return L - 1; }, p.scale_log2 * pools.k_scale[kv_head],
             pools.v_scale[kv_head]);
  uint32_t at = 0;
  auto take = [&](auto nb, int j) {
    constexpr int NB = decltype(nb)::value;
    const uint8_t* t[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      t[i] = ring + at;
      at = at == (S - 1) * Tile<HD>::kBytes ? 0 : at + Tile<HD>::kBytes;
    }
    wait_copies<S - NB>();
    rows.template blocks<NB, true>(t, j * kBS, L - j * kBS);
    __syncwarp();
#pragma unroll 1
    for (int i = 0; i < NB; ++i) feed();
  };
  int i = 0;
  for (; i + RowsT::TAKE <= n; i += RowsT::TAKE)
    take(std::integral_constant<int, RowsT::TAKE>{}, j0 + i);
  if (RowsT::TAKE > 2 && i + 2 <= n) {
    take(std::integral_constant<int, 2>{}, j0 + i);
    i += 2;
  }
  if (RowsT::TAKE > 1 && i < n) take(std::integral_constant<int, 1>{}, j0 + i);
  T* out = static_cast<T*>(p.out) + (int64_t(b) * p.n_heads + int64_t(grp) * rows_per_group) * HD;
  if (C == 1) {
    rows.store([&](int r) -> T* { return r < p.rep ? out + (warp * p.rep + r) * HD : nullptr; });
    return;
  }
  // this CTA's part
  rows.store_partial(
      [&](int r) -> float* { return r < p.rep ? part_o + r * HD : nullptr; },
      [&](int r) -> float* { return part_ml + (warp * p.rep + r) * 2; });

  cluster_sync();  // every CTA's partial is in its shared memory
  // CTA `rank` combines float4s [rank E / C, (rank + 1) E / C) of the group's E
  const int per_warp = p.rep * HD / 4;
  const int E = p.hg_size * per_warp;
  const int e0 = rank * E / C, e1 = (rank + 1) * E / C;
  for (int e = e0 + static_cast<int>(threadIdx.x); e < e1; e += static_cast<int>(blockDim.x)) {
    const int r = e / (HD / 4), w = e / per_warp;
    const float* o_at = reinterpret_cast<const float*>(smem + w * room) + (e - w * per_warp) * 4;
    float2 ml[kMaxCluster];
    float4 oc[kMaxCluster];
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {  // every peer's values in one round trip
      ml[c] = make_float2(0.f, 0.f);
      oc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < C) {
        ml[c] = ld_cluster_f32x2(cluster_map(part_ml + r * 2, c));
        oc[c] = ld_cluster_f32x4(cluster_map(o_at, c));
      }
    }
    float M = -INFINITY;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c)
      if (ml[c].y > 0.f) M = fmaxf(M, ml[c].x);  // a part that saw no key has no weight
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
      if (ml[c].y > 0.f) {
        const float w = fast_exp2(ml[c].x - M) * ml[c].y;
        den += w;
        acc = make_float4(fmaf(w, oc[c].x, acc.x), fmaf(w, oc[c].y, acc.y), fmaf(w, oc[c].z, acc.z),
                          fmaf(w, oc[c].w, acc.w));
      }
    }
    const float inv = den > 0.f ? 1.f / den : 0.f;
    store4(out + e * 4, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  }
  cluster_sync();  // the peers have read this CTA's partials
}

// Joins for batches of few groups, which many CTAs share (a single long sequence: all of
// them): a CTA is 32 float4 of one group's rows, its warps share the parts, eight loads of
// each on their way, and join their sums through shared memory.  (One thread for all the
// parts of its element, as joins of two or three parts go, took 55 us of the 62 for one
// sequence of 8,192 tokens.)
constexpr int kWideJoin = 8;  // warps
constexpr int kFewParts = 16;  // CTAs a group, from which on

template <typename T, int HD>
__global__ void __launch_bounds__(kWideJoin * 32) join_few_kernel(const DecodeParams p) {
  constexpr int NB = 8;  // parts on their way
  __shared__ float4 sum_s[kWideJoin][32];
  __shared__ float2 ml_s[kWideJoin][32];
  attn::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (the lengths were there before the decode began)
  const int b = blockIdx.x / p.n_groups, grp = blockIdx.x - b * p.n_groups;
  const WarpScan scan(p);
  const int2 seq = scan.of(b);
  // the decode's partials; and a CTA that ends without the wait would let this grid, and so
  // the kernel after it, run ahead of the decode
  attn::pdl_wait();
  const int U = scan.total, G = p.grid;
  const int nblk = seq.y / p.n_groups;
  if (nblk == 0) return;
  const int first = seq.x + grp * nblk;
  const int c0 = owner_of(first, U, G), c1 = owner_of(first + nblk - 1, U, G);
  if (c0 == c1) return;  // not split
  // c0 holds the group's first units at the end of its range, unless its range starts there
  const bool tail = attn::range_begin(c0, U, G) != first;
  const int rows = p.hg_size * p.rep;
  const int E = rows * HD;  // elements of a part
  const int e = (blockIdx.y * 32 + lane) * 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, den = 0.f;
  if (e < E) {
    for (int cs = c0 + warp; cs <= c1; cs += NB * kWideJoin) {
      float4 o[NB];
      float2 ml[NB];
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int c = cs + k * kWideJoin;
        o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        ml[k] = make_float2(-INFINITY, 0.f);
        // (with fewer units than CTAs some ranges are empty)
        if (c <= c1 && (U >= G || attn::range_begin(c + 1, U, G) > attn::range_begin(c, U, G))) {
          const int64_t slot = 2 * c + (c == c0 && tail ? 1 : 0);
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
  }
  sum_s[warp][lane] = acc;
  ml_s[warp][lane] = make_float2(M, den);
  __syncthreads();
  if (warp != 0 || e >= E) return;
#pragma unroll
  for (int w = 1; w < kWideJoin; ++w) {
    const float2 ml = ml_s[w][lane];
    const float4 o = sum_s[w][lane];
    if (ml.y > 0.f) {
      const float Mn = fmaxf(M, ml.x);
      const float a = fast_exp2(M - Mn), f = fast_exp2(ml.x - Mn);
      acc = make_float4(fmaf(f, o.x, acc.x * a), fmaf(f, o.y, acc.y * a), fmaf(f, o.z, acc.z * a),
                        fmaf(f, o.w, acc.w * a));
      den = fmaf(den, a, f * ml.y);
      M = Mn;
    }
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  const float4 v = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  T* out = static_cast<T*>(p.out) + (int64_t(b) * p.n_heads + int64_t(grp) * rows) * HD + e;
  store4(out, v);
}

// --------------------------------------------------------------- host side

template <typename T, int HD, int NT>
struct DecodeFp4 {
  static constexpr int kCtas = kCtasPerSm<T, HD, NT>;
  static constexpr int kDepth = kStages<T, HD, NT>;
  static_assert(kDepth > Rows<T, HD, NT, false>::TAKE, "blocks at hand and on their way");
  static size_t ring_bytes(int warps, int nstages) {
    return (size_t(warps) * nstages * Tile<HD>::kBytes + 127) / 128 * 128;
  }

  static cudaError_t run(const AttnArgs& a, const Fp4Cache& cache, cudaStream_t stream) {
    const PoolShape& pool = a.pool;
    const Pools pools(cache);
    DecodeParams p{};
    p.q = a.q;
    p.out = a.out;
    p.bt = a.block_tables;
    p.seq_lens = a.seq_lens;
    p.err = a.err;
    p.B = a.num_seqs;
    p.n_heads = a.n_heads;
    p.n_kv = pool.n_kv;
    p.rep = a.n_heads / pool.n_kv;
    p.W = a.max_blocks_per_seq;
    p.num_blocks = pool.num_blocks;
    p.max_len = a.max_seq_len;  // (no more than the tables hold)
    p.max_seq_len = a.max_seq_len;
    p.head_dim = HD;
    p.scale_log2 = a.scale * attn::kLog2e;
    const int hg = head_group(pool.n_kv);
    p.hg_size = hg;
    p.n_groups = pool.n_kv / hg;
    // (narrow groups have many CTAs an SM, and read lengths again)
    const size_t kept = hg >= 4 ? kKeptLens * 4 : 0;
    const size_t smem = ring_bytes(hg, kDepth) + kept;
    static KernelSetup setup;
    int per_sm = 0;
    cudaError_t e = kernel_setup(setup, decode_kernel<T, HD, NT>, static_cast<int>(smem), hg * 32,
                                 &per_sm, kSmemMax);
    if (e != cudaSuccess) return e;
    per_sm = std::max(1, std::min(per_sm, 16));  // 16: what the workspace is sized for
    int G = sm_count() * per_sm;
    if (a.max_ctas > 0 && a.max_ctas < G) G = a.max_ctas;
    const int nmax = p.max_len / kBS + (p.max_len % kBS != 0);
    const int64_t max_units = int64_t(a.num_seqs) * p.n_groups * nmax;
    // (parts of four blocks at the least: one sequence of 4,096 tokens of 8 x 128 takes 10.4
    // us so, in parts of one block 17.1, of eight 12.4)
    const int part = a.max_ctas > 0 ? 1 : 4;
    if (max_units < int64_t(part) * G) G = static_cast<int>(std::max<int64_t>(1, max_units / part));
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
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;

    // Batches of sequences that a cluster can take whole.  A block takes a warp about the
    // same time (0.55 us at 64, 0.75 at 128) whether it has an SM for itself or shares it
    // with fifteen others (it is its chain of dependent steps), so the fewer a warp has the
    // better: as many CTAs to a sequence as the GPU runs at once, but one where that is at
    // most two steps for its warps.  A stream shares the blocks out evenly, but pays some 6
    // us for its scan, its partial results and its join (9 where groups are narrow): so
    // clusters as long as their warps have few blocks more, if all sequences were of the
    // longest length.  64 sequences of 8 x 64, 32 heads: of 128 tokens 5.4 us (two CTAs each
    // 5.9, streamed 10.7), of 512 9.3 (14.1), of 2,048 23.6 (26.2); 20 of 4,096 22.5 (21.3);
    // 700 of 512 tokens of 8 x 128, 64 heads, one CTA each, 84 (92); 16 of 4,096 35.9 (29.8);
    // 11 of 1,211 of 3 x 64, 9 heads, 6.8 (13.0); 46 of 2,202 of 3 x 128 18.3 (16.3).
    const int slots = sm_count() * per_sm;
    const int64_t groups = int64_t(a.num_seqs) * p.n_groups;
    int C = nmax <= 8 ? 1 : std::min(kMaxCluster, (nmax + 3) / 4);
    // (clusters lie within GPCs, which leaves up to a tenth of the SMs' places empty, where
    // an SM holds one CTA and clusters are of 7 or 8 a quarter)
    auto fits = [&](int c) {
      return groups * c * 20 <= int64_t(slots) * (c < 7 ? 18 : per_sm < 2 ? 13 : c == 7 ? 17 : 18);
    };
    while (C > 1 && !fits(C)) --C;
    const int blocks = std::max(1, (nmax + C - 1) / C);  // a warp's
    // (than an even share)
    const int64_t shares = std::max<int64_t>(1, std::min<int64_t>(slots, max_units));
    const int more = blocks - static_cast<int>(max_units / shares);
    const int most = HD == 128 ? 9 : hg < 4 ? 16 : 12;
    if (a.max_ctas == 0 && blocks <= kMaxBlocks && more <= most) {
      p.cluster = C;
      p.nstages = (std::max(std::min(kDepth, blocks) * Tile<HD>::kBytes, p.rep * HD * 4) + 127) / 128 * 128;
      p.part_off = hg * p.nstages;
      const size_t need = p.part_off + (size_t(hg) * p.rep * 2 * 4 + 15) / 16 * 16;
      static KernelSetup cluster_setup;
      e = kernel_setup(cluster_setup, decode_cluster_kernel<T, HD, NT>, kSmemMax, kWarps * 32, nullptr);
      if (e != cudaSuccess) return e;
      attr[1].id = cudaLaunchAttributeClusterDimension;
      attr[1].val.clusterDim.x = static_cast<unsigned>(C);
      attr[1].val.clusterDim.y = 1;
      attr[1].val.clusterDim.z = 1;
      cfg.numAttrs = 2;
      cfg.gridDim = dim3(static_cast<unsigned>(groups * C));
      cfg.blockDim = dim3(hg * 32);
      cfg.dynamicSmemBytes = need;
      e = cudaLaunchKernelEx(&cfg, decode_cluster_kernel<T, HD, NT>, p, pools);
      return e != cudaSuccess ? e : cudaGetLastError();
    }
    p.nstages = kDepth;
    p.part_off = kept != 0 ? static_cast<int>(ring_bytes(hg, kDepth)) : 0;  // the kept lengths
    // every CTA scans the lengths in its stages; larger batches have a plan kernel
    p.plan_in_kernel =
        a.num_seqs <= 32 * kLaneSeqs ||
        (a.num_seqs <= kKernelPlanSeqs &&
         size_t(a.num_seqs + 1 + 32) * 4 <= size_t(hg) * kDepth * Tile<HD>::kBytes);
    if (!p.plan_in_kernel) {
      attn::decode_plan_kernel<T, HD><<<1, 1024, 0, stream>>>(p);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    cfg.gridDim = dim3(G);
    cfg.blockDim = dim3(hg * 32);
    cfg.dynamicSmemBytes = smem;
    e = cudaLaunchKernelEx(&cfg, decode_kernel<T, HD, NT>, p, pools);
    if (e != cudaSuccess) return e;
    const int vecs = hg * p.rep * HD / 4;  // of a group's rows
    cfg.dynamicSmemBytes = 0;
    if (p.B <= 32 * kLaneSeqs && int64_t(p.B) * p.n_groups * kFewParts <= G) {
      cfg.gridDim = dim3(p.B * p.n_groups, (vecs + 31) / 32);
      cfg.blockDim = dim3(kWideJoin * 32);
      e = cudaLaunchKernelEx(&cfg, join_few_kernel<T, HD>, p);
      return e != cudaSuccess ? e : cudaGetLastError();
    }
    const int threads = std::min(fp8::kJoinThreads, (vecs + 31) / 32 * 32);
    cfg.gridDim = dim3(G, (vecs + threads - 1) / threads);
    cfg.blockDim = dim3(threads);
    e = cudaLaunchKernelEx(&cfg, fp8::join_kernel<T, HD>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
};

template <typename T>
cudaError_t decode_as(const AttnArgs& a, const Fp4Cache& c, cudaStream_t s) {
  const bool one = a.n_heads / a.pool.n_kv <= 8;
  switch (a.pool.head_dim) {
    case 16: return one ? DecodeFp4<T, 16, 1>::run(a, c, s) : DecodeFp4<T, 16, 2>::run(a, c, s);
    case 32: return one ? DecodeFp4<T, 32, 1>::run(a, c, s) : DecodeFp4<T, 32, 2>::run(a, c, s);
    case 64: return one ? DecodeFp4<T, 64, 1>::run(a, c, s) : DecodeFp4<T, 64, 2>::run(a, c, s);
    default: return one ? DecodeFp4<T, 128, 1>::run(a, c, s) : DecodeFp4<T, 128, 2>::run(a, c, s);
  }
}

// The two output types are compiled in their own translation units.
cudaError_t decode_fp4_bf16(const AttnArgs& a, const Fp4Cache& c, cudaStream_t s);
cudaError_t decode_fp4_f32(const AttnArgs& a, const Fp4Cache& c, cudaStream_t s);

}  // namespace fp4
}  // namespace pkv
