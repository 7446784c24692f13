// Chunked prefill over the 4-bit cache on warp-level tensor cores: fp32 queries, and
// bf16 queries of narrow heads (mathematics and tile layouts in fp4_rows.cuh).
//
// CTA = (query tile, KV head, sequence).  Eight consumer warps each own 16 / rep
// consecutive queries x all rep query heads of the KV head; a producer lane streams
// the head's blocks into a ring that all of them read, up to the tile's last visible
// key.  Bound by the consumers' conversions and products: each warp turns the block's
// codes into f16 for itself.  4 chunks of 256 at the end of 1,000 tokens, 8 heads on 4: fp32
// 49 us at head_dim 64 and 89 at 128, where the registers do not hold two row tiles with
// their second terms (168 bytes a thread stored to local memory, 116 read); bf16 27 us at 16
// and 29 at 32 (there, with two CTAs an SM, 8 and 32 bytes).
#pragma once

#include "attention.cuh"
#include "decode_fp4.cuh"

namespace pkv {
namespace fp4 {

using attn::PrefillParams;
using attn::Ring;
using attn::kBarrierBytes;
using fp8::RingPos;
using fp8::gave_up;
using fp8::release_tile;

constexpr int kPrefillWarps = 8;
constexpr int kPrefillTiles = 2;  // row tiles of 8 per warp
constexpr int kPrefillRows = 8 * kPrefillTiles;

// Producer, one lane (elect_one): fetches blocks into the ring one after the other.
template <int HD>
struct Producer {
  const Ring& ring;
  const Pools& pools;
  int num_blocks, n_kv, head;
  int32_t* err;
  RingPos pos;
  uint32_t issued = 0;

  // The head's part of block `id`; a bad one reads zeros.  False on timeout.
  __device__ __forceinline__ bool fetch(int id) {
    if (pos.round > 0 && !wait_or_abort(ring.empty + pos.st, (pos.round - 1) & 1, ring.abort_flag)) {
      report(err, PKV_DEVERR_TIMEOUT);
      return false;
    }
    uint8_t* t = ring.k_tile(pos.st);
    uint64_t* full = ring.full + pos.st;
    using TileT = Tile<HD>;
    if (id >= 0 && id < num_blocks) {
      mbar_arrive_expect_tx(full, TileT::kBytes);
      const int64_t at = int64_t(id) * n_kv + head;
      // (the chunk's other tiles read the blocks again: no eviction hint)
      bulk_copy_g2s(t, pools.k + at * TileT::kCodes, TileT::kCodes, full);
      bulk_copy_g2s(t + TileT::kVCodes, pools.v + at * TileT::kCodes, TileT::kCodes, full);
      bulk_copy_g2s(t + TileT::kKGroups, pools.kg + at * TileT::kGroups, TileT::kGroups, full);
      bulk_copy_g2s(t + TileT::kVGroups, pools.vg + at * TileT::kGroups, TileT::kGroups, full);
    } else {
      report(err, PKV_DEVERR_BLOCK_ID);
      // scales of zero: whatever codes the stage holds are then zeros
      for (int i = 0; i < 2 * TileT::kGroups; i += 16)
        *reinterpret_cast<uint4*>(t + TileT::kKGroups + i) = make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async_smem();  // before the copies that come there next
      mbar_arrive(full);
    }
    pos.next(ring);
    ++issued;
    return true;
  }

  // Blocks row[0 .. n), ids read a group ahead.  False: gave up (and told the consumers).
  __device__ __forceinline__ bool fetch_row(const int32_t* row, int n) {
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
        if (!fetch(id[i])) {
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
  if (use) rows.template blocks<NB, true>(t, j0, valid);
#pragma unroll
  for (int i = 0; i < NB; ++i) release_tile(ring, at[i]);
}

// CTAS: that an SM's registers hold.
template <typename T, int HD, int CTAS>
__global__ void __launch_bounds__((kPrefillWarps + 1) * 32, CTAS)
    prefill_kernel(const PrefillParams p, const Pools pools, const ChunkLimits limits,
                   const int last_seq) {
  extern __shared__ __align__(128) uint8_t smem[];
  attn::pdl_wait();
  attn::pdl_launch_dependents();
  const int b = blockIdx.z;
  const int g = blockIdx.y;
  const int q0 = p.cu_q[b], end = p.cu_q[b + 1];
  if (threadIdx.x == 0 && blockIdx.x == 0 && g == 0)
    report_bad_chunk(p.err, limits, q0, end, p.seq_lens[b], b == last_seq);
  if (q0 < 0 || end <= q0 || end > p.total_q) return;  // no chunk, or not within the rows
  const int c = end - q0;
  const int tile_q = kPrefillWarps * p.queries_per_warp;
  const int64_t first = int64_t(blockIdx.x) * tile_q;
  if (first >= c) return;  // whole CTA idle: exit before touching barriers
  const int i0 = static_cast<int>(first);
  const int L = min(p.seq_lens[b], p.max_len);
  if (L < c) return;  // inconsistent chunk: nothing computed
  const int i_end = min(c, i0 + tile_q);
  const int n_blocks = (L - c + i_end - 1) / kBS + 1;  // up to the last key any row sees

  Ring ring = attn::make_tile_ring(smem, p.nstages, Tile<HD>::kBytes / 2);
  attn::ring_init(ring, kPrefillWarps);
  const int warp = threadIdx.x >> 5;
  const int32_t* row = p.bt + int64_t(b) * p.W;

  if (warp == kPrefillWarps) {
    if (elect_one()) {
      Producer<HD> pr{ring, pools, p.num_blocks, p.n_kv, g, p.err};
      pr.fetch_row(row, n_blocks);
      pr.finish();
    }
  } else {
    using RowsT = Rows<T, HD, kPrefillTiles, true>;
    RowsT rows;
    rows.place();
    const T* q = static_cast<const T*>(p.q);
    const int qw = i0 + warp * p.queries_per_warp;  // first query of this warp
    const int nrows = p.queries_per_warp * p.rep;
    auto query_of = [&](int r) { return qw + r / p.rep; };
    auto head_of = [&](int r) { return g * p.rep + r % p.rep; };
    rows.begin(
        [&](int r) -> const T* {
          if (r >= nrows || query_of(r) >= c) return nullptr;
          return q + (int64_t(q0 + query_of(r)) * p.n_heads + head_of(r)) * HD;
        },
        [&](int r) { return L - c + query_of(r); }, p.scale_log2 * pools.k_scale[g], pools.v_scale[g]);
    // this warp's last visible key
    const int my_last = qw < c ? L - c + min(c, qw + p.queries_per_warp) - 1 : -1;
    RingPos pos;
    for (int k = 0; k < n_blocks;) {
      if ((k & 31) == 0 && gave_up(ring)) break;
      const int j0 = k * kBS;
      const bool use = j0 <= my_last;
      if (RowsT::PAIR == 2 && k + 1 < n_blocks) {
        take_tiles<RowsT::PAIR>(rows, ring, pos, j0, L - j0, use, p.err);
        k += RowsT::PAIR;
      } else {
        take_tiles<1>(rows, ring, pos, j0, L - j0, use, p.err);
        ++k;
      }
    }
    if (!gave_up(ring)) {
      T* out = static_cast<T*>(p.out);
      rows.store([&](int r) -> T* {
        if (r >= nrows || query_of(r) >= c) return nullptr;
        return out + (int64_t(q0 + query_of(r)) * p.n_heads + head_of(r)) * HD;
      });
    }
  }
}

template <typename T, int HD>
cudaError_t prefill_run(const AttnArgs& a, const Fp4Cache& cache, cudaStream_t stream) {
  const PoolShape& pool = a.pool;
  const Pools pools(cache);
  PrefillParams p{};
  p.q = a.q;
  p.out = a.out;
  p.bt = a.block_tables;
  p.seq_lens = a.seq_lens;
  p.cu_q = a.cu_q_lens;
  p.err = a.err;
  p.B = a.num_seqs;
  p.n_heads = a.n_heads;
  p.n_kv = pool.n_kv;
  p.rep = a.n_heads / pool.n_kv;
  p.W = a.max_blocks_per_seq;
  p.num_blocks = pool.num_blocks;
  p.max_len = a.max_seq_len;  // (no more than the tables hold)
  p.total_q = a.total_q;
  p.scale_log2 = a.scale * attn::kLog2e;
  p.queries_per_warp = kPrefillRows / p.rep;
  p.nstages = 12;
  const size_t smem = kBarrierBytes + 1024 + size_t(p.nstages) * Tile<HD>::kBytes;
  const int tile_q = kPrefillWarps * p.queries_per_warp;
  const int64_t tiles = (int64_t(a.max_q_len) + tile_q - 1) / tile_q;
  if (tiles == 0 || a.num_seqs == 0) return cudaSuccess;
  auto kern = prefill_kernel<T, HD, 1>;
  int ctas = 1;
  if constexpr (sizeof(T) == 2) {
    // CTAs with work: each sequence may have one tile that is not full
    const int64_t busy =
        std::min(tiles * a.num_seqs, int64_t(a.total_q) / tile_q + a.num_seqs) * pool.n_kv;
    if (busy > sm_count()) {
      kern = prefill_kernel<T, HD, 2>;
      ctas = 2;
    }
  }
  static KernelSetup setup[2];
  const int threads = (kPrefillWarps + 1) * 32;
  cudaError_t e = kernel_setup(setup[ctas - 1], kern, static_cast<int>(smem), threads, nullptr);
  if (e != cudaSuccess) return e;
  const ChunkLimits limits{a.total_q, a.max_q_len, a.max_seq_len,
                           int64_t(a.max_blocks_per_seq) * kBS};
  // the grid's y and z extents are 16-bit: long batches go in slices
  for (int s0 = 0; s0 < a.num_seqs; s0 += 65535) {
    PrefillParams ps = p;
    ps.B = std::min(65535, a.num_seqs - s0);
    ps.cu_q += s0;
    ps.seq_lens += s0;
    ps.bt += int64_t(s0) * p.W;
    const dim3 grid(static_cast<unsigned>(tiles), pool.n_kv, ps.B);
    const int last_seq = s0 + ps.B == a.num_seqs ? ps.B - 1 : -1;
    e = launch_pdl(kern, grid, threads, smem, stream, ps, pools, limits, last_seq);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace fp4
}  // namespace pkv
