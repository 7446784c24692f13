// Decode over the 4-bit cache: one query per sequence attends to the sequence's pages
// (mathematics and layouts of the tiles in fp4_rows.cuh).
//
// Bound by reading the cache: 9 / 8 x n_kv x head_dim bytes a token.  The work split is
// that of the 8-bit decode: a persistent grid over equal contiguous ranges of
// (sequence, head group, block) units, a joining kernel for the groups that several
// CTAs share, and one thread-block cluster per (sequence, head group) for batches too
// small to stream.  A head's rows of a block lie together in the pools, so a block of
// a group's heads is four contiguous runs (K and V, codes and scales: 18 KB at 8 heads
// of 128) that one producer lane fetches with bulk copies; one consumer warp per KV
// head.
#pragma once

#include "attention.cuh"
#include "decode_fp8.cuh"
#include "fp4_rows.cuh"

namespace pkv {
namespace fp4 {

using attn::DecodeParams;
using attn::DecodeWs;
using attn::Ring;
using attn::kBarrierBytes;
using attn::kKernelPlanSeqs;
using attn::kMaxCluster;
using attn::kMaxStages;
using fp8::RingPos;
using fp8::Walk;
using fp8::gave_up;
using fp8::head_group;
using fp8::kKeptLens;
using fp8::length_of;
using fp8::release_tile;
using fp8::report_bad_length;

constexpr int kMaxThreads = 9 * 32;

__device__ __forceinline__ void bulk_copy_hint(void* dst, const void* src, uint32_t bytes,
                                               uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1], %2, [%3], %4;" ::"r"(smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

// The pools as the producer reads them.
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

__device__ __forceinline__ Ring make_ring(uint8_t* smem, int nstages, int stage_bytes) {
  Ring r = attn::make_tile_ring(smem, nstages, stage_bytes / 2);
  return r;
}

// Producer, one lane (elect_one): fetches blocks into the ring one after the other.
template <int HD>
struct Producer {
  const Ring& ring;
  const Pools& pools;
  int num_blocks, n_kv, heads;  // heads: of a tile
  int32_t* err;
  uint64_t policy;  // nonzero: an L2 cache policy for the copied lines
  RingPos pos;
  uint32_t issued = 0;

  // Heads head0 .. of block `id`; a bad one reads zeros.  False on timeout.
  __device__ __forceinline__ bool fetch(int id, int head0) {
    if (pos.round > 0 && !wait_or_abort(ring.empty + pos.st, (pos.round - 1) & 1, ring.abort_flag)) {
      report(err, PKV_DEVERR_TIMEOUT);
      return false;
    }
    uint8_t* t = ring.k_tile(pos.st);
    uint64_t* full = ring.full + pos.st;
    const uint32_t codes = heads * kBS * HD / 2, groups = heads * kBS * HD / kGroup;
    if (id >= 0 && id < num_blocks) {
      mbar_arrive_expect_tx(full, 2 * (codes + groups));
      const int64_t row = (int64_t(id) * n_kv + head0) * kBS;
      copy(t, pools.k + row * (HD / 2), codes, full);
      copy(t + codes, pools.v + row * (HD / 2), codes, full);
      copy(t + 2 * codes, pools.kg + row * (HD / kGroup), groups, full);
      copy(t + 2 * codes + groups, pools.vg + row * (HD / kGroup), groups, full);
    } else {
      report(err, PKV_DEVERR_BLOCK_ID);
      // scales of zero: whatever codes the stage holds are then zeros
      for (uint32_t i = 0; i < 2 * groups; i += 16)
        *reinterpret_cast<uint4*>(t + 2 * codes + i) = make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async_smem();  // before the copies that come there next
      mbar_arrive(full);
    }
    pos.next(ring);
    ++issued;
    return true;
  }

  __device__ __forceinline__ void copy(void* dst, const void* src, uint32_t bytes, uint64_t* bar) const {
    if (policy != 0) bulk_copy_hint(dst, src, bytes, bar, policy);
    else bulk_copy_g2s(dst, src, bytes, bar);
  }

  // Blocks row[0 .. n), ids read a group ahead.  False: gave up (and told the consumers).
  __device__ __forceinline__ bool fetch_row(const int32_t* row, int n, int head0) {
    constexpr int kAhead = 8;
    int id[kAhead], next[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) next[i] = i < n ? row[i] : 0;
    for (int k0 = 0; k0 < n; k0 += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) id[i] = next[i];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) next[i] = k0 + kAhead + i < n ? row[k0 + kAhead + i] : 0;
      if (*ring.abort_flag) return false;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (k0 + i >= n) break;
        if (!fetch(id[i], head0)) {
          *ring.abort_flag = 1;
          return false;
        }
      }
    }
    return true;
  }

  // At the end: until the consumers have left the last tile, and all have landed; where
  // some thread gave up, a bounded wait for the copies still in flight, so that none
  // lands after the CTA has left.
  __device__ __forceinline__ void finish() const {
    if (issued == 0) return;
    const uint32_t last = issued - 1, st = last % ring.nstages;
    const bool left = wait_or_abort(ring.empty + st, (last / ring.nstages) & 1, ring.abort_flag);
    if (!left || *ring.abort_flag) attn::ring_drain(ring, issued);
  }
};

// Consumer warp: its next NB tiles of the ring.  After a wait that gave up the warp goes
// on over what is there (its work is all its lanes'); gave_up tells before anything is
// stored.
template <int NB, typename RowsT>
__device__ __forceinline__ void take_tiles(RowsT& rows, const Ring& ring, RingPos& pos, int j0,
                                           int valid, bool use, int32_t* err) {
  const uint8_t* t[NB];
  RingPos at[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    at[i] = pos;
    t[i] = ring.k_tile(pos.st);
    wait_or_flag(ring.full + pos.st, pos.round & 1, ring.abort_flag, err);
    pos.next(ring);
  }
  if (use) rows.template blocks<NB>(t, j0, valid);
#pragma unroll
  for (int i = 0; i < NB; ++i) release_tile(ring, at[i]);
}

// CTAs of 8 consumer warps that an SM's registers hold.
template <typename T, int HD, int NT>
constexpr int kCtasPerSm = NT == 1 && HD * int(sizeof(T)) / 2 <= 128 ? 2 : 1;

template <typename T, int HD, int NT, int CTAS>
__global__ void __launch_bounds__(kMaxThreads, CTAS)
    decode_kernel(const DecodeParams p, const Pools pools) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int consumers = p.hg_size;
  Ring ring = make_ring(smem, p.nstages, Tile::bytes(p.hg_size, HD));
  attn::ring_init(ring, consumers);
  attn::pdl_wait();               // inputs and workspace belong to the preceding kernel
  attn::pdl_launch_dependents();  // the merge kernel may be scheduled (it waits for this grid)

  const int warp = threadIdx.x >> 5;
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
      Producer<HD> pr{ring, pools, p.num_blocks, p.n_kv, p.hg_size, p.err, tc::l2_evict_first_policy()};
      bool ok = true;
      for (int u = r0; u < r1 && ok;) {
        const int n = min(r1 - u, cur.nblk - cur.j);
        ok = pr.fetch_row(p.bt + int64_t(cur.b) * p.W + cur.j, n, cur.grp * p.hg_size);
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
    using RowsT = Rows<T, HD, NT, false>;
    RowsT rows;
    rows.place(p.hg_size, warp);
    RingPos pos;
    const T* q = static_cast<const T*>(p.q);
    T* out = static_cast<T*>(p.out);
    for (int u = r0; u < r1;) {
      const int n = min(r1 - u, cur.nblk - cur.j);
      const int b = cur.b;
      const int kv_head = cur.grp * p.hg_size + warp;
      const int head0 = kv_head * p.rep;
      const int last = cur.L - 1;
      rows.begin(
          [&](int r) -> const T* {
            return r < p.rep ? q + (int64_t(b) * p.n_heads + head0 + r) * HD : nullptr;
          },
          [&](int) { return last; }, p.scale_log2 * pools.k_scale[kv_head], pools.v_scale[kv_head]);
      for (int k = 0; k < n;) {
        if ((k & 31) == 0 && gave_up(ring)) break;
        const int j0 = (cur.j + k) * kBS;
        if (RowsT::PAIR == 2 && k + 1 < n) {
          take_tiles<RowsT::PAIR>(rows, ring, pos, j0, cur.L - j0, true, p.err);
          k += RowsT::PAIR;
        } else {
          take_tiles<1>(rows, ring, pos, j0, cur.L - j0, true, p.err);
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

// Batches too small to stream: one cluster of C CTAs per (sequence, head group), each a
// contiguous part of the sequence's at most 8 * C blocks, the parts combined through
// distributed shared memory (as the 8-bit decode's cluster path; no workspace, no merge
// launch).
template <typename T, int HD, int NT>
__global__ void __launch_bounds__(kMaxThreads, 1)
    decode_cluster_kernel(const DecodeParams p, const Pools pools) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int consumers = p.hg_size;
  Ring ring = make_ring(smem, p.nstages, Tile::bytes(p.hg_size, HD));
  attn::ring_init(ring, consumers);
  const int warp = threadIdx.x >> 5;
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
  const int L = length_of(p, b);
  const int nblk = (L + kBS - 1) / kBS;
  const int j0 = rank * nblk / C, j1 = (rank + 1) * nblk / C;
  if (blockIdx.x == 0 && threadIdx.x == 0)
    p.total_units[1] = -1;  // a call planning for itself replaces any kept plan
  if (rank == 0 && grp == 0 && threadIdx.x == 0) report_bad_length(p, b);

  uint32_t issued = 0;
  if (warp == consumers) {
    if (elect_one()) {
      Producer<HD> pr{ring, pools, p.num_blocks, p.n_kv, p.hg_size, p.err, tc::l2_evict_first_policy()};
      pr.fetch_row(p.bt + int64_t(b) * p.W + j0, j1 - j0, grp * p.hg_size);
      issued = pr.issued;
    }
  } else if (warp < consumers) {
    using RowsT = Rows<T, HD, NT, false>;
    const T* q = static_cast<const T*>(p.q);
    const int kv_head = grp * p.hg_size + warp;
    const int head0 = kv_head * p.rep;
    RowsT rows;
    rows.place(p.hg_size, warp);
    rows.begin(
        [&](int r) -> const T* {
          return r < p.rep ? q + (int64_t(b) * p.n_heads + head0 + r) * HD : nullptr;
        },
        [&](int) { return L - 1; }, p.scale_log2 * pools.k_scale[kv_head], pools.v_scale[kv_head]);
    RingPos pos;
    for (int j = j0; j < j1;) {
      const int jp = j * kBS;
      if (RowsT::PAIR == 2 && j + 1 < j1) {
        take_tiles<RowsT::PAIR>(rows, ring, pos, jp, L - jp, true, p.err);
        j += RowsT::PAIR;
      } else {
        take_tiles<1>(rows, ring, pos, jp, L - jp, true, p.err);
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

// --------------------------------------------------------------- host side

template <typename T, int HD, int NT>
struct DecodeFp4 {
  static constexpr int kSmemMax = 226 * 1024;  // what both kernels opt in to
  static int stage_bytes(int hg) { return Tile::bytes(hg, HD); }
  // barriers, alignment slack and ring; what follows starts there
  static size_t smem_for(int hg, int nstages) {
    return kBarrierBytes + 1024 + size_t(nstages) * stage_bytes(hg);
  }
  static constexpr int kDoubled = kCtasPerSm<T, HD, NT>;
  // Ring depth: about 176 KB of stages per SM, shared by the CTAs of 8 consumer warps
  // in all (narrow groups: several CTAs per SM, each with its barriers and kept
  // lengths).
  static int ring_stages(int hg) {
    const int ctas = std::max(1, 8 / hg) * kDoubled;
    const int ns = (176 - 4 * (ctas - 1)) * 1024 / ctas / stage_bytes(hg);
    return std::max(2, std::min(kMaxStages, ns));
  }
  static cudaError_t grid(const AttnArgs& a, int hg, int* G, size_t* smem, int* nstages, int* wave) {
    *nstages = ring_stages(hg);
    *smem = smem_for(hg, *nstages) + kKeptLens * 4;
    static KernelSetup setup;
    int per_sm = 0;
    const cudaError_t e = kernel_setup(setup, decode_kernel<T, HD, NT, kDoubled>, static_cast<int>(*smem),
                                       (hg + 1) * 32, &per_sm, kSmemMax);
    if (e != cudaSuccess) return e;
    per_sm = std::max(1, std::min(per_sm, 16));  // 16: what the workspace is sized for
    *G = sm_count() * per_sm;
    *wave = *G / kDoubled;
    if (a.max_ctas > 0 && a.max_ctas < *G) *G = a.max_ctas;
    const int64_t max_units = int64_t(a.num_seqs) * (a.pool.n_kv / hg) *
                              ((int64_t(a.max_seq_len) + kBS - 1) / kBS);
    if (max_units < *G) *G = static_cast<int>(std::max<int64_t>(1, max_units));
    return cudaSuccess;
  }

  static cudaError_t run(const AttnArgs& a, const Fp4Cache& cache, cudaStream_t stream) {
    const PoolShape& pool = a.pool;
    const Pools pools(cache);
    const int hg = head_group(pool.n_kv);
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
    p.hg_size = hg;
    p.n_groups = pool.n_kv / hg;
    p.W = a.max_blocks_per_seq;
    p.num_blocks = pool.num_blocks;
    p.max_len = a.max_seq_len;  // (no more than the tables hold)
    p.max_seq_len = a.max_seq_len;
    p.head_dim = HD;
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
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3((hg + 1) * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;

    // Latency-bound batches, by the rule of the bf16 decode: the longest sequence at
    // most 64 blocks and the clusters within two waves.
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
      e = kernel_setup(setup, decode_cluster_kernel<T, HD, NT>, kSmemMax, (hg + 1) * 32, nullptr);
      if (e != cudaSuccess) return e;
      attr[1].id = cudaLaunchAttributeClusterDimension;
      attr[1].val.clusterDim.x = static_cast<unsigned>(C);
      attr[1].val.clusterDim.y = 1;
      attr[1].val.clusterDim.z = 1;
      cfg.numAttrs = 2;
      cfg.gridDim = dim3(static_cast<unsigned>(ctas));
      cfg.dynamicSmemBytes = p.part_off + extra;
      e = cudaLaunchKernelEx(&cfg, decode_cluster_kernel<T, HD, NT>, p, pools);
      return e != cudaSuccess ? e : cudaGetLastError();
    }
    p.part_off = static_cast<int>(smem_for(hg, p.nstages));  // the kept lengths
    // every CTA scans the lengths in its ring stages; larger batches have a plan kernel
    p.plan_in_kernel = a.num_seqs <= kKernelPlanSeqs &&
                       size_t(a.num_seqs + 1 + 32) * 4 <= size_t(p.nstages) * stage_bytes(hg);
    if (!p.plan_in_kernel) {
      attn::decode_plan_kernel<T, HD><<<1, 1024, 0, stream>>>(p);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    cfg.gridDim = dim3(G);
    cfg.dynamicSmemBytes = smem;
    e = cudaLaunchKernelEx(&cfg, decode_kernel<T, HD, NT, kDoubled>, p, pools);
    if (e != cudaSuccess) return e;
    const int vecs = hg * p.rep * HD / 4;  // of a group's rows
    const int threads = std::min(fp8::kJoinThreads, (vecs + 31) / 32 * 32);
    cfg.gridDim = dim3(G, (vecs + threads - 1) / threads);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = 0;
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
