// Eviction: of each sequence with more than keep_tiles full tiles, the tiles
// with the least mass leave the block table.
//
// The unit is the tile: its tokens share the channel factors C and its pages
// are shared by all KV heads, so a tile leaves whole, without requantizing.
// Attention does not depend on the order of the cached tokens (the rows carry
// their positions), but the order of the tiles is kept: the kept ones move up
// in order, the evicted ones' blocks follow them, and later blocks stay, so a
// row stays a permutation of itself and the next tiles that the sequence
// fills reuse the evicted blocks.  The raw tail stays where it is (a row's
// place in it is its position mod T, and lengths shrink by multiples of T).
//
// One CTA per sequence.  The masses as unsigned keys in their order; the e-th
// smallest free key by three histogram passes of 11, 11 and 10 bits; equal
// keys leave by index; one scan gives every tile its new place.  Bound by the
// latency of these steps, not by the bytes: up to kSmallTiles tiles the keys
// and the new order stay in shared memory, and up to kHeld blocks a thread the
// row is moved through registers.  Longer rows go through the workspace.
#include <cuda_runtime.h>

#include "kvq_device.cuh"

namespace kvq {

namespace {

constexpr int kThreads = 1024;
constexpr int kSmallTiles = 4096;  // keys and order in shared memory up to here
constexpr int kHeld = 16;          // blocks of a row a thread can hold
constexpr int kBins = 2048;

// workspace per sequence: new order of the tiles, staged blocks, staged masses
struct EvictWs {
  size_t order, blocks, mass, stride;  // in 32-bit words
};
__host__ __device__ inline EvictWs evict_ws(int max_blocks, int pages_per_tile) {
  EvictWs w;
  const size_t tiles = static_cast<size_t>(max_blocks) / pages_per_tile;
  w.order = 0;
  w.blocks = w.order + tiles;
  w.mass = w.blocks + max_blocks;
  w.stride = w.mass + tiles;
  return w;
}

// unsigned key in the order of the masses: -0 equals 0, NaN comes last
__device__ __forceinline__ uint32_t mass_key(float x) {
  const uint32_t u = __float_as_uint(x);
  if (x != x) return 0xffffffffu;
  if (x == 0.f) return 0x80000000u;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// exclusive scan of a flag over the CTA; `total` gets the sum
__device__ __forceinline__ int block_scan(bool flag, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned bal = __ballot_sync(kFull, flag);
  __syncthreads();  // the last scan's totals have been read
  if (lane == 0) s_warp[warp] = __popc(bal);
  __syncthreads();
  const int w = s_warp[lane];  // 32 warps
  total = __reduce_add_sync(kFull, w);
  const int before = __reduce_add_sync(kFull, lane < warp ? w : 0);
  return before + __popc(bal & ((1u << lane) - 1u));
}

__global__ void __launch_bounds__(kThreads, 1) evict_kernel(EvictArgs a) {
  __shared__ uint32_t s_key[kSmallTiles];
  __shared__ int s_order[kSmallTiles];
  __shared__ int s_hist[kBins];
  __shared__ int s_warp[32];
  __shared__ int s_digit, s_need;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int T = a.cfg.tile_tokens, ppt = T / kPageTokens, page_bits = ppt == 2 ? 1 : (ppt == 4 ? 2 : 3);
  float* mass = a.mass + static_cast<size_t>(b) * a.max_tiles;
  int32_t* table = a.block_tables + static_cast<size_t>(b) * a.max_blocks_per_seq;
  int32_t* kept = a.kept ? a.kept + static_cast<size_t>(b) * a.max_tiles : nullptr;
  const EvictWs wl = evict_ws(a.max_blocks_per_seq, ppt);
  int32_t* ws = static_cast<int32_t*>(a.workspace) + b * wl.stride;

  const int len = max(a.seq_lens[b], 0), n = len / T;
  const bool bad = n > a.max_blocks_per_seq / ppt || n > a.max_tiles;
  if (bad && tid == 0) report_error(a.dev_status, KVQ_ERR_DEVICE_BOUNDS);
  const int gone = bad ? 0 : max(0, n - a.keep_tiles), left = n - gone;
  if (kept != nullptr && (bad || gone == 0))
    for (int i = tid; i < a.max_tiles; i += kThreads) kept[i] = !bad && i < n ? i : -1;
  if (gone == 0) return;
  const bool small = n <= kSmallTiles;
  int32_t* order = small ? s_order : ws + wl.order;
  if (small)
    for (int i = tid; i < n; i += kThreads) s_key[i] = mass_key(mass[i]);
  auto key = [&](int i) { return small ? s_key[i] : mass_key(mass[i]); };
  const float tail = n < a.max_tiles ? mass[n] : 0.f;

  // the gone-th smallest key among the free tiles, digit by digit
  const int f0 = a.sink_tiles, f1 = n - a.recent_tiles;
  uint32_t prefix = 0, mask = 0;
  int need = gone;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t digits = pass == 2 ? 1023u : 2047u;
    s_hist[tid] = 0;
    s_hist[tid + kThreads] = 0;
    __syncthreads();
    for (int i = f0 + tid; i < f1; i += kThreads) {
      const uint32_t k = key(i);
      if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & digits], 1);
    }
    __syncthreads();
    // thread t: bins 2t and 2t + 1 behind `before` keys
    const int c0 = s_hist[2 * tid], c1 = s_hist[2 * tid + 1];
    int incl = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    const int before = incl - c0 - c1 + __reduce_add_sync(kFull, lane < warp ? s_warp[lane] : 0);
    if (before < need && need <= before + c0 + c1) {  // one thread
      const bool second = need > before + c0;
      s_digit = 2 * tid + second;
      s_need = need - before - (second ? c0 : 0);
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_digit) << shift;
    mask |= digits << shift;
    need = s_need;
  }
  // keys below `prefix` leave, and the first `need` equal to it; a tile's new
  // place from the scans
  int ties = 0, out = 0;  // before this round of tiles
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + tid;
    const bool free_tile = i >= f0 && i < f1;
    const uint32_t k = free_tile ? key(i) : 0u;
    int total;
    const int tie = ties + block_scan(free_tile && k == prefix, s_warp, total);
    ties += total;
    const bool leaves = free_tile && (k < prefix || (k == prefix && tie < need));
    const int gone_before = out + block_scan(leaves, s_warp, total);
    out += total;
    if (i < n) order[leaves ? left + gone_before : i - gone_before] = i;
  }
  __syncthreads();
  // the row and the masses, read whole before they are written
  const int blocks = n << page_bits;
  auto source = [&](int i) { return (order[i >> page_bits] << page_bits) + (i & (ppt - 1)); };
  if (small && blocks <= kHeld * kThreads) {
    int32_t held[kHeld];
    float moved[kSmallTiles / kThreads];
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (tid + k * kThreads < blocks) held[k] = table[source(tid + k * kThreads)];
#pragma unroll
    for (int k = 0; k < kSmallTiles / kThreads; ++k)
      if (tid + k * kThreads < left) moved[k] = mass[order[tid + k * kThreads]];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (tid + k * kThreads < blocks) table[tid + k * kThreads] = held[k];
#pragma unroll
    for (int k = 0; k < kSmallTiles / kThreads; ++k)
      if (tid + k * kThreads < left) mass[tid + k * kThreads] = moved[k];
  } else {
    int32_t* staged = ws + wl.blocks;
    float* moved = reinterpret_cast<float*>(ws + wl.mass);
    for (int i = tid; i < blocks; i += kThreads) staged[i] = table[source(i)];
    for (int i = tid; i < left; i += kThreads) moved[i] = mass[order[i]];
    __syncthreads();
    for (int i = tid; i < blocks; i += kThreads) table[i] = staged[i];
    for (int i = tid; i < left; i += kThreads) mass[i] = moved[i];
  }
  for (int i = left + tid; i < a.max_tiles; i += kThreads) mass[i] = i == left ? tail : 0.f;
  if (kept != nullptr)
    for (int i = tid; i < a.max_tiles; i += kThreads) kept[i] = i < left ? order[i] : -1;
  if (tid == 0) a.seq_lens[b] = len - gone * T;
}

}  // namespace

size_t evict_workspace_bytes(const kvq_config& cfg, int num_seqs, int max_blocks_per_seq) {
  return static_cast<size_t>(num_seqs) * evict_ws(max_blocks_per_seq, cfg.tile_tokens / kPageTokens).stride *
         sizeof(int32_t);
}

cudaError_t launch_evict_tiles(const EvictArgs& a, cudaStream_t s) {
  evict_kernel<<<a.num_seqs, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
