// Chunked prefill over the 8-bit cache on warp-level tensor cores: fp32
// queries, and bf16 queries of narrow heads (mathematics and tile layouts in
// fp8_rows.cuh).
//
// CTA = (query tile, KV head, sequence).  Eight consumer warps each own
// 16 / rep consecutive queries x all rep query heads of the KV head; a producer
// lane streams the head's blocks (16 tokens x head_dim bytes of K and V) into
// a ring that all of them read, up to the tile's last visible key.  Bound by
// the consumers' conversions and products: each warp turns the block's e4m3
// values into f16 for itself.  Measured, 4 chunks of 256 at the end of 1,000
// tokens, 32 heads on 8: fp32 96 us at head_dim 64 (76 TFLOP/s) and 146 us at
// 128 (which spills 272 bytes a thread), bf16 46 us at head_dim 32.
#pragma once

#include "attention.cuh"
#include "decode_fp8.cuh"

namespace pkv {
namespace fp8 {

using attn::PrefillParams;

constexpr int kPrefillWarps = 8;
constexpr int kPrefillTiles = 2;  // row tiles of 8 per warp
constexpr int kPrefillRows = 8 * kPrefillTiles;

// CTAS: that an SM's registers hold.  Two, at 96 registers, hide each other's
// latencies, but each is slower: for bf16 (narrow heads), where there are more CTAs
// than SMs (when it was chosen: 4 chunks of 256 at the end of 1,000 tokens, 32
// heads of 32 on 8: 46.4 us in place of 58.5; 6 chunks of 37, 8 heads of 16 on 4:
// 9.5 and 8.9).  fp32 would spill several times what it does (4 chunks as above,
// heads of 128: 251 us for 163).
template <typename T, int HD, int CTAS>
__global__ void __launch_bounds__((kPrefillWarps + 1) * 32, CTAS)
    prefill_kernel(const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const PrefillParams p,
                   const Scales sc, const ChunkLimits limits, const int last_seq) {
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
  const int i0 = blockIdx.x * tile_q;
  if (i0 >= c) return;  // whole CTA idle: exit before touching barriers
  const int L = min(p.seq_lens[b], p.max_len);
  if (L < c) return;  // inconsistent chunk: nothing computed
  const int i_end = min(c, i0 + tile_q);
  const int n_blocks = (L - c + i_end - 1) / kBS + 1;  // up to the last key any row sees

  Ring ring = attn::make_tile_ring(smem, p.nstages, kBS * HD);
  attn::ring_init(ring, kPrefillWarps);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t* row = p.bt + int64_t(b) * p.W;

  if (warp == kPrefillWarps) {
    if (elect_one()) {  // (the chunk's other tiles read the blocks again: no eviction hint)
      Producer pr{ring, &tm_k, &tm_v, p.num_blocks, p.err, 0};
      pr.fetch_row(row, n_blocks, g);
      pr.finish();
    }
  } else {
    Rows<T, HD, kPrefillTiles, true> rows;
    rows.place(HD, 0);
    const T* q = static_cast<const T*>(p.q);
    const int qw = i0 + warp * p.queries_per_warp;  // first query of this warp
    const int nrows = p.queries_per_warp * p.rep;
    auto query_of = [&](int r) { return qw + r / p.rep; };
    auto head_of = [&](int r) { return g * p.rep + r % p.rep; };
    DecodeParams dp{};  // what a scale batch needs of the pool
    dp.num_blocks = p.num_blocks;
    dp.n_kv = p.n_kv;
    auto id_at = [&](int i) { return i < n_blocks ? row[i] : -1; };
    ScaleBatch now, next;
    next.load(sc, dp, id_at(lane), g);
    int ids = id_at(32 + lane);
    rows.begin(
        [&](int r) -> const T* {
          if (r >= nrows || query_of(r) >= c) return nullptr;
          return q + (int64_t(q0 + query_of(r)) * p.n_heads + head_of(r)) * HD;
        },
        [&](int r) { return L - c + query_of(r); }, p.scale_log2);
    // this warp's last visible key
    const int my_last = qw < c ? L - c + min(c, qw + p.queries_per_warp) - 1 : -1;
    RingPos pos;
    constexpr int PAIR = Rows<T, HD, kPrefillTiles, true>::PAIR;
    for (int k = 0; k < n_blocks;) {
      if ((k & 31) == 0) {
        if (gave_up(ring)) break;
        now = next;
        now.settle();
        next.load(sc, dp, ids, g);
        ids = id_at(k + 64 + lane);
      }
      const int j0 = k * kBS;
      const bool use = j0 <= my_last;
      if (PAIR == 2 && k + 1 < n_blocks) {
        take_tiles<PAIR>(rows, ring, pos, now, k, j0, L - j0, use, p.err);
        k += PAIR;
      } else {
        take_tiles<1>(rows, ring, pos, now, k, j0, L - j0, use, p.err);
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
cudaError_t prefill_run(const AttnArgs& a, const Scales& sc, cudaStream_t stream) {
  const PoolShape& pool = a.pool;
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
  const size_t smem = kBarrierBytes + 1024 + size_t(p.nstages) * 2 * kBS * HD;
  CUtensorMap tm_k{}, tm_v{};
  if (!encode_tiles(&tm_k, a.k_pool, pool, HD, 1) || !encode_tiles(&tm_v, a.v_pool, pool, HD, 1))
    return cudaErrorInvalidValue;
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
    e = launch_pdl(kern, grid, threads, smem, stream, tm_k, tm_v, ps, sc, limits, last_seq);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace fp8
}  // namespace pkv
