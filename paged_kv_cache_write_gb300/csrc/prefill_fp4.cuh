// Chunked prefill over the 4-bit cache on warp-level tensor cores: fp32 queries, and
// bf16 queries of narrow heads (mathematics and tile layouts in fp4_rows.cuh).
//
// CTA = (query tile, KV head, sequence).  Eight consumer warps each own 16 / rep
// consecutive queries x all rep query heads of the KV head; a producer lane streams
// the head's blocks into a ring that all of them read, up to the tile's last visible
// key.  Bound by the consumers' conversions and products: each warp turns the block's
// codes into f16 for itself.
#pragma once

#include "attention.cuh"
#include "decode_fp4.cuh"

namespace pkv {
namespace fp4 {

using attn::PrefillParams;

constexpr int kPrefillWarps = 8;
constexpr int kPrefillTiles = 2;  // row tiles of 8 per warp
constexpr int kPrefillRows = 8 * kPrefillTiles;

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

  Ring ring = make_ring(smem, p.nstages, Tile::bytes(1, HD));
  attn::ring_init(ring, kPrefillWarps);
  const int warp = threadIdx.x >> 5;
  const int32_t* row = p.bt + int64_t(b) * p.W;

  if (warp == kPrefillWarps) {
    if (elect_one()) {  // (the chunk's other tiles read the blocks again: no eviction hint)
      Producer<HD> pr{ring, pools, p.num_blocks, p.n_kv, 1, p.err, 0};
      pr.fetch_row(row, n_blocks, g);
      pr.finish();
    }
  } else {
    using RowsT = Rows<T, HD, kPrefillTiles, true>;
    RowsT rows;
    rows.place(1, 0);
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
  const size_t smem = kBarrierBytes + 1024 + size_t(p.nstages) * Tile::bytes(1, HD);
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
