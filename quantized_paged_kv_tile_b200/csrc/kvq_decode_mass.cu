// Paged decode attention that adds the attention weight of every tile to its
// mass: the decode of kvq_decode_kernel.cuh with per-tile statistics, then
// one pass over them.
//
//   mass[b][t] += sum over query heads h of  l_t,h exp2(m_t,h - M_h) / L_h
//
// with l_t,h the sum of tile t's weights relative to the running maximum
// m_t,h it had, and M_h, L_h the head's final maximum and sum.  The statistics
// are 8 bytes per (tile, query head) against the tile's 9216 bytes per KV head
// (T = 64, 4-bit codes).  6 sequences of 131073 tokens, 8 x 4 heads: 310 us in a
// graph against 285 without masses.  21 of the 25 are in the tile kernel (a second
// running sum, two shuffles and a store a tile, in code that is bound by issue
// slots), 4 in the pass below.
#include "kvq_decode_kernel.cuh"
#include "kvq_launch.cuh"

namespace kvq {

namespace {

template <int T, int BK, int BV>
struct MassLauncher {
  static cudaError_t run(const DecodeArgs& a, cudaStream_t s, int sms) {
    return launch_decode_bits<T, BK, BV, true>(a, s, sms);
  }
};

// A warp per kMassTilesPerWarp tiles, lanes over the query heads; the heads of
// a lane in order, then the lanes by butterfly, so the sum has one fixed order.
// The tiles' reads are in flight together: the pass is bound by their latency.
constexpr int kMassTilesPerWarp = 8;
constexpr int kMassWarps = 4;
__global__ void __launch_bounds__(kMassWarps * 32) decode_mass_kernel(DecodeArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.y, T = a.cfg.tile_tokens, hqn = a.cfg.num_kv_heads * a.cfg.group_size;
  cudaGridDependencySynchronize();
  const int tiles = (max(a.seq_lens[b], 0) + T - 1) / T;
  const int served = min(tiles, min(a.mass_tiles, a.mass_stat_tiles));
  if (blockIdx.x == 0 && threadIdx.x == 0 && served < tiles) report_error(a.dev_status, KVQ_ERR_DEVICE_BOUNDS);
  const int t0 = (blockIdx.x * kMassWarps + warp) * kMassTilesPerWarp;
  if (t0 >= served) return;
  const float2* fin = a.mass_final + static_cast<size_t>(b) * hqn;
  const float2* st = a.mass_stats + (static_cast<size_t>(b) * a.mass_stat_tiles + t0) * hqn;
  float* out = a.mass + static_cast<size_t>(b) * a.mass_tiles + t0;
  const float old = lane < kMassTilesPerWarp && t0 + lane < served ? out[lane] : 0.f;
  float sum[kMassTilesPerWarp];
#pragma unroll
  for (int k = 0; k < kMassTilesPerWarp; ++k) sum[k] = 0.f;
  for (int h = lane; h < hqn; h += 32) {
    const float2 f = fin[h];
    float2 x[kMassTilesPerWarp];
#pragma unroll
    for (int k = 0; k < kMassTilesPerWarp; ++k)
      x[k] = t0 + k < served ? st[static_cast<size_t>(k) * hqn + h] : make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kMassTilesPerWarp; ++k)
      if (x[k].x != 0.f) sum[k] += x[k].x * exp2f(x[k].y - f.x) * f.y;  // an empty share has no maximum
  }
  float mine = 0.f;
#pragma unroll
  for (int k = 0; k < kMassTilesPerWarp; ++k) {
    const float s = warp_sum(sum[k]);
    if (lane == k) mine = s;
  }
  if (lane < kMassTilesPerWarp && t0 + lane < served) out[lane] = old + mine;
}

size_t stats_offset(const kvq_config& cfg, int num_seqs, int num_splits, int sms) {
  return (decode_workspace_bytes(cfg, num_seqs, num_splits, sms) + 255) / 256 * 256;
}

}  // namespace

int decode_mass_stat_tiles(const kvq_config& cfg, int max_blocks_per_seq) {
  return max_blocks_per_seq / (cfg.tile_tokens / kPageTokens) + 1;  // the table's tiles and the raw tail
}

size_t decode_mass_workspace_bytes(const kvq_config& cfg, int num_seqs, int max_blocks_per_seq, int num_splits,
                                   int sms) {
  const size_t heads = static_cast<size_t>(num_seqs) * cfg.num_kv_heads * cfg.group_size;
  return stats_offset(cfg, num_seqs, num_splits, sms) +
         heads * (static_cast<size_t>(decode_mass_stat_tiles(cfg, max_blocks_per_seq)) + 1) * sizeof(float2);
}

cudaError_t launch_paged_decode_mass(DecodeArgs a, cudaStream_t s) {
  if (a.num_seqs == 0) return cudaSuccess;
  const int sms = device_sms();
  const size_t heads = static_cast<size_t>(a.num_seqs) * a.cfg.num_kv_heads * a.cfg.group_size;
  a.mass_stat_tiles = decode_mass_stat_tiles(a.cfg, a.max_blocks_per_seq);
  a.mass_final = reinterpret_cast<float2*>(static_cast<char*>(a.workspace) +
                                           stats_offset(a.cfg, a.num_seqs, a.num_splits_fixed, sms));
  a.mass_stats = a.mass_final + heads;
  cudaError_t e;
  if (a.cfg.head_dim != kHeadDim) {
    e = launch_generic_decode(a, s);
  } else {
    switch (a.cfg.tile_tokens) {
      case 32: e = dispatch_decode_bits<32, MassLauncher>(a, s, sms); break;
      case 64: e = dispatch_decode_bits<64, MassLauncher>(a, s, sms); break;
      default: e = dispatch_decode_bits<128, MassLauncher>(a, s, sms); break;
    }
  }
  if (e != cudaSuccess) return e;
  const int per_cta = kMassTilesPerWarp * kMassWarps;
  const int tiles = std::min(a.mass_tiles, a.mass_stat_tiles);
  return launch_behind(decode_mass_kernel, dim3((tiles + per_cta - 1) / per_cta, a.num_seqs), kMassWarps * 32, s, a);
}

}  // namespace kvq
