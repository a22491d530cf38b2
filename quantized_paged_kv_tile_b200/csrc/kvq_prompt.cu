// Read path, whole prompts: causal attention over raw fp16 rows, packed
// sequences of different lengths, grouped heads.
//
// Query token i of a sequence (query head j, KV head j / g) sees the keys of
// tokens 0..i of its sequence:
//   out_i = sum_j p_ij v_j,  p_ij = exp(c q_i.k_j - lse_i),
//   lse_i = ln sum_{j <= i} exp(c q_i.k_j).
// One pass over the keys with the running maximum m and sum l of the softmax
// in the log2 domain (c log2 e folded into the exponent's multiply-add).
//
// A query tile is 128 rows, one per TMEM lane: tokens x the g query heads of a
// KV head, token-major.  A work unit is (sequence, run of one or two query
// tiles, KV head).  One persistent CTA per SM takes units longest first, in two
// streams (one at d = 256): a query tile each, or, where there are few units,
// half of the keys of one query tile each, merged by their log-sum-exp at the
// end.  Its warps pass tiles on through mbarriers:
//   unit warp      finds the CTA's units and publishes them; as V guard it
//                  cleans the V tiles that masks reach into
//   load warp      TMA: the unit's Q tiles, then K and V tiles through a ring
//   MMA warps      (one per stream) S = Q K^T and O += P V, tcgen05, fp32
//                  in TMEM, P as A operand from TMEM, V as it lies in memory
//                  (keys as rows: an MN-major B operand)
//   softmax warps  (four per stream, a row per thread) S from TMEM, running
//                  maximum and sum in registers, P as fp16 to TMEM, O rescaled
//                  where the maximum moved far; at the end O / l to memory
// P is rounded to fp16 (half a step is 2^-11 of each weight; for those below
// 2^-14 of the row's largest 2^-25 of that, or less where the keys are many, see
// spare_bits; the sum l takes the unrounded weights), everything else stays in
// fp32.
//
// What bounds it: at d = 128 a pair of 128 x 128 tiles needs 2048 cycles of
// the tensor pipe and 2186 of the exponential unit (measured: 128 exponentials
// a thread take two warps of a scheduler that long) and takes about 3300, the
// chain P -> P V -> Q K^T -> S -> maximum -> exponentials of a query tile; long
// calls run into the power limit first (1567 MHz at 1000 W; a library fp16
// GEMM of 8192^3 settles at 1287 TFLOP/s there, this kernel at 1030 to 1100).
// 16384 tokens x 64 heads: K channels of one std 3.44 ms in five calls (1279
// TFLOP/s) and 4.01 in 400; of very different stds, whose scores move the
// maximum further, 3.76 and 4.29.  Replacing 1/8 to 3/8 of the exponentials by a
// polynomial on the FMA pipe gained 1.6% on short runs and lost 4 to 11% on long
// ones.
//
// What a mask hides never reaches a result: masked scores become -inf by
// selection; V rows past the sequence are zeroed in shared memory; V values
// of the tiles that straddle the diagonal that are not finite are replaced
// by zero there and added, unweighted, to exactly the rows that see them.
//
// Mass (optional): per row and run of T keys the sum of the weights, with the
// maximum it is relative to, goes to a scratch area of the CTA; once a query
// tile's l and m are final, the rows that count are weighted and summed, and a
// second kernel adds the query tiles of a sequence to its masses in a fixed
// order.  It costs a sixth of the attention (4 x 4096 tokens, 32 heads: 542 us
// without, 626 with all queries counting).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kvq_device.cuh"
#include "kvq_launch.cuh"
#include "kvq_sm100.cuh"

namespace kvq {

namespace {

using namespace sm100;

constexpr int kRows = 128;    // query rows per query tile (TMEM lanes)
// The running maximum a row's weights are relative to follows the true one
// only once that is more than kLazy larger (log2 units): weights reach 2^15
// then, below fp16's 65504 and held by it and the fp32 sums as exactly as 1.
// A rescale of O costs a warp about as much as a tile's exponentials; with
// keys of very different channel stds (scores spread over some 30 units) a
// limit of 8 took 4853 us on 16384 tokens x 64 heads.
constexpr float kLazy = 15.f;
// Scaled scores (log2 units) from here on count as infinite, those below the
// negative as -inf.  The exponent's multiply-add rounds once, the scaled
// maximum that it subtracts before: up to here by half a unit at most, all of a
// row's weights alike, which l cancels; further out that would take them out of
// fp16's range.  (A score has no bits below one left there.)
constexpr float kFar = 16777216.f;  // 2^24
// When the maximum moves, a weight of 2^spare goes to the score it moves to, so
// that small weights are rounded as late.  A weight is rounded to a multiple of
// fp16's smallest, 2^-24, at worst: off by 2^-25 of 2^-spare of the row's
// largest, and over `keys` keys by less than 2^-12 of it (half a step of an
// fp16 output is 2^-12 to 2^-11 of that).  Every bit spared leaves kLazy one
// less: up to 8192 keys none is needed, 2 at 32768, 7 at 2^20 (us without and
// with, spread scores: 16384 tokens x 64 heads 3838 / 3899, 131072 x 4 14990 /
// 15280; d = 64, 32768 x 16: 2886 / 2881).
__device__ __forceinline__ float spare_bits(int keys) { return static_cast<float>(max(0, 19 - __clz(keys - 1))); }
// up to this many sequences the units are taken longest first
constexpr int kSortedSeqs = 1024;

struct PromptDev {
  PromptArgs a;
  int tile_tokens;     // query tokens per query tile
  int unit_tokens;     // query tokens per unit (one or two query tiles), W
  uint32_t unit_magic; // floor(2^32 / W) + 1: the high word of x times it is x / W for x < 2^24
  int units;           // host bound on the number of units
  int max_tiles_k;     // key tiles of the longest sequence
  int window_runs;     // query tiles per (sequence, head) that can hold counted queries; 0: all
  float qscale;        // softmax_scale * log2 e
  float* scratch;      // per CTA and query tile [max_tiles_k][entries per key tile + 1][kRows]
  float* part;         // per query tile of the call [max_tiles_k * entries per key tile]
};

// whether rows [first, end) can be a sequence
__device__ __forceinline__ bool seq_ok(int first, int end, int total, int longest) {
  return first >= 0 && end >= first && end <= total && end - first <= longest;
}
// Length and first row of sequence s; 0 tokens if the prefix sums are bad.
__device__ __forceinline__ int seq_len(const PromptArgs& a, int s, int& first) {
  first = a.cu_seqlens[s];
  const int end = a.cu_seqlens[s + 1];
  return seq_ok(first, end, a.total_tokens, a.max_seq_tokens) ? end - first : 0;
}

struct Unit {
  int seq, run, head, n, first;  // n = 0: nothing here
};

// Finds the units; one warp uses it, all lanes together.  Only sequences before
// the first descent of the prefix sums have any: behind it they could overlap
// earlier ones, and the units would be more than the host counted.
// Up to kSortedSeqs sequences: units in descending order of their run index
// (so of their keys), from a binary search over the levels, count(c) = number
// of runs >= c.  Up to 32 sequences their run counts stay in registers, a lane
// each (a search took 4000 to 5000 cycles with loads and divisions in it).
// More: sequence s owns the slots from first_s / W + s on, found by binary
// search; slots past its units are empty.
class UnitFinder {
 public:
  // (the numbers are copied: read through a reference to the kernel's
  // arguments each cost a trip through memory)
  // `ascending`: sequences before the first descent, where there are more than 32
  __device__ UnitFinder(const PromptDev& pd, int ascending, int lane)
      : cu_(pd.a.cu_seqlens), seqs_(pd.a.num_seqs), total_(pd.a.total_tokens), longest_(pd.a.max_seq_tokens),
        heads_(pd.a.cfg.num_kv_heads), W_(pd.unit_tokens), magic_(pd.unit_magic), lane_(lane) {
    int f;
    if (seqs_ > 32) {
      seqs_ = ascending;
    } else {
      const unsigned down = __ballot_sync(kFull, lane < seqs_ && cu_[lane + 1] < cu_[lane]);
      if (down != 0) seqs_ = __ffs(down) - 1;
    }
    if (lane < seqs_) mine_ = runs(len(lane, f));
  }

  __device__ Unit find(int u) const {
    const int x = u / heads_;
    Unit r{0, 0, u - x * heads_, 0, 0};
    if (seqs_ > kSortedSeqs) {
      int lo = 0, hi = seqs_;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (max(cu_[mid], 0) / W_ + mid <= x) lo = mid; else hi = mid;
      }
      int f = 0;
      const int n = len(lo, f);
      r.run = x - (f / W_ + lo);
      if (r.run >= 0 && r.run < runs(n)) {
        r.seq = lo;
        r.n = n;
        r.first = f;
      }
      return r;
    }
    if (count(0) <= x) return r;
    int lo = 0, hi = runs(longest_), above = 0;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1, k = count(mid);
      if (k > x) {
        lo = mid;
      } else {
        hi = mid;
        above = k;
      }
    }
    int k = x - above;  // the k-th sequence that has a run `lo`
    for (int s0 = 0; s0 < seqs_; s0 += 32) {
      const bool mine = runs_of(s0 + lane_) > lo;
      const unsigned has = __ballot_sync(kFull, mine);
      const unsigned at = __ballot_sync(kFull, mine && __popc(has & ((1u << lane_) - 1u)) == k);
      if (at != 0) {
        r.seq = s0 + __ffs(at) - 1;
        r.run = lo;
        r.n = len(r.seq, r.first);
        return r;
      }
      k -= __popc(has);
    }
    return r;
  }

 private:
  __device__ int len(int s, int& first) const {
    first = cu_[s];
    const int end = cu_[s + 1];
    return seq_ok(first, end, total_, longest_) ? end - first : 0;
  }
  // ceil(n / W), n <= 2^20
  __device__ int runs(int n) const { return __umulhi(static_cast<uint32_t>(n + W_ - 1), magic_); }
  __device__ int runs_of(int s) const {
    int f;
    if (seqs_ <= 32) return s == lane_ ? mine_ : 0;
    return s < seqs_ ? runs(len(s, f)) : 0;
  }
  __device__ int count(int c) const {
    int k = 0;
    if (seqs_ <= 32)
      k = max(0, mine_ - c);
    else
      for (int s = lane_; s < seqs_; s += 32) k += max(0, runs_of(s) - c);
    return __reduce_add_sync(kFull, k);
  }
  const int32_t* cu_;
  int seqs_, total_, longest_, heads_, W_;
  uint32_t magic_;
  int lane_, mine_ = 0;
};

// slot of query tile `run` of u's sequence and head in the partial masses; -1:
// none of its queries counts
__device__ __forceinline__ long long mass_slot(const PromptDev& pd, const Unit& u, int run) {
  const PromptArgs& a = pd.a;
  const int W1 = pd.tile_tokens;
  if (a.mass_window == 0) return (static_cast<long long>(u.first / W1 + u.seq + run)) * a.cfg.num_kv_heads + u.head;
  const int r0 = max(0, u.n - a.mass_window) / W1;
  if (run < r0) return -1;
  return (static_cast<long long>(u.seq) * pd.window_runs + (run - r0)) * a.cfg.num_kv_heads + u.head;
}

// max that keeps NaN
__device__ __forceinline__ float max3nan(float x, float y, float z) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// max of magnitudes, NaN left out
__device__ __forceinline__ float max3abs(float x, float y, float z) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// Shapes per head size.  kQT query tiles of 128 rows share the key tiles that
// the CTA loads.  Each has its own softmax warpgroup, its own warp that issues
// its matrix instructions, and its own score, P and output tiles in TMEM.
// At d = 64 and 256 P has columns of its own, so the next scores can be
// computed as soon as the softmax has read the last ones.  At d = 128 the two
// output tiles leave no room for that: P lies over S.
template <int D, bool MASS>
struct Geom {
  static constexpr int kQT = D == 256 ? 1 : 2;
  static constexpr bool kOver = D == 128;               // P over S
  static constexpr int kKeys = D == 256 ? 64 : 128;     // keys per tile
  // With P over S a query tile waits for its MMAs between P and the next
  // scores: the two softmaxes take turns at the exponentials, so that one's
  // MMAs run under the other's exponentials (left alone they drift into step:
  // 1171 against 1218 TFLOP/s).  Where nothing waits, turns only cost (d = 64:
  // 608 against 654).
  static constexpr bool kTurns = kOver;
  static constexpr int kSlot = kKeys * D * 2;                                  // one K or V tile
  static constexpr int kSlots = D == 64 ? 8 : 4;
  static constexpr int kThreads = kQT * 128 + 128;      // softmax; two MMA warps, loads, V guard and units
  static constexpr int kQTile = kRows * D * 2;
  static constexpr int kQ = 0;
  static constexpr int kKV = kQ + kQT * kQTile;
  static constexpr int kStat = kKV + kSlots * kSlot;    // float m[128], w[128] per query tile (masses)
  static constexpr int kStage = kStat + kQT * 2 * kRows * 4;  // per softmax warp 32 rows x 32 channels fp16
  static constexpr int kBar = kStage + kQT * 4 * 2048;
  static constexpr int kMisc = kBar + 384;
  static constexpr int kSmem = kMisc + 128 + 1024;      // + alignment slack
  static_assert(kSmem <= 232448, "shared memory per block");
  // TMEM columns: S and P of query tile q from q * kTile on, O after them
  static constexpr int kTile = D == 64 ? 192 : 128;
  static constexpr int kO = kQT * kTile;
  static constexpr int kP = kOver ? 0 : kKeys;
  static_assert((kOver ? kKeys : kKeys + kKeys / 2) <= kTile && kO + kQT * D <= 512, "TMEM columns");
};

// mbarriers, 8 bytes each, from Geom::kBar on; [q]: one per query tile
constexpr int kUnitSlots = 4;
enum : int {
  kBarQFull = 0,             // the unit's Q tiles have landed
  kBarQEmpty,                // the last score MMAs have read them
  kBarS,                     // [q] a score tile is in TMEM
  kBarF = kBarS + 2,         // [q] the softmax has read it (one arrival per warp)
  kBarH = kBarF + 2,         // [q] the first half of its P is in TMEM (one arrival per warp)
  kBarI = kBarH + 2,         // [q] three quarters are
  kBarP = kBarI + 2,         // [q] all of it is
  kBarO = kBarP + 2,         // [q] its P V is done
  kBarT = kBarO + 2,         // [q] query tile q's turn at the exponentials
  kBarM = kBarT + 2,         // SPLIT: [1] stream 1 is done with a unit, [0] stream 0 has merged it
  kBarUFull = kBarM + 2,     // [unit slot] a unit is published
  kBarUEmpty = kBarUFull + kUnitSlots,  // [unit slot] every warp is done with it
  kBarDrain = kBarUEmpty + kUnitSlots,  // [q]
  kBarKVFull = kBarDrain + 2,           // [slot] a K or V tile has landed
  kBarKVEmpty = kBarKVFull + 8,         // [slot] every MMA that reads it is done
  kBarCount = kBarKVEmpty + 8
};
static_assert(kBarCount * 8 <= 384, "barriers fit");

struct Shared {  // at Geom::kMisc
  uint32_t tmem;
  int stop;
  int edges, guarded;     // edge tiles, in all, whose V is on its way / that the V guard is done with
  int ascending;          // more than 32 sequences: those before the first descent of the prefix sums
  int odd_v[kUnitSlots];  // per unit: V values of an edge tile were left out
  Unit unit[kUnitSlots];
};
static_assert(sizeof(Shared) <= 128, "shared words fit");

// A running position in a ring of barriers
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n, int base = 0) {  // n slots from base on
    if (++slot == base + n) {
      slot = base;
      phase ^= 1u;
    }
  }
};

// Counters in shared memory, for what may run several steps ahead of its
// waiter (a barrier's parity would then be ambiguous).  Wait, a whole warp,
// until the counter has reached `n`; bounded like the barriers' waits.
__device__ __forceinline__ void set_count(int* counter, int n) {
  __threadfence_block();
  *static_cast<volatile int*>(counter) = n;
}
__device__ __forceinline__ bool wait_count(const volatile int* counter, int n, volatile int* stop) {
  if (__all_sync(kFull, *counter >= n)) {
    __threadfence_block();
    return true;
  }
  const long long t0 = global_ns();
  bool ok = true;
  while (ok && *counter < n) {
    if (global_ns() - t0 > kWaitLimitNs) *stop = 1;
    ok = !*stop;
  }
  __threadfence_block();
  return __all_sync(kFull, ok);
}

// What stream q of a CTA (its MMA warp, its softmax warpgroup, its columns of
// TMEM) does of a unit that starts at token i0: the key tiles [lo, hi) for the
// query tile that starts at token `first`.  Usually a stream has a query tile
// of its own; in SPLIT launches a unit is one query tile and the two streams
// share out its key tiles, to be merged at the end.
struct Work {
  int first, lo, hi;
  __device__ __forceinline__ int count() const { return hi - lo; }
};
template <int KT, bool SPLIT>
__device__ __forceinline__ Work stream_work(int i0, int q, int W1, int n) {
  const int first = i0 + (SPLIT ? 0 : q * W1);
  const int tiles = first < n ? (min(n, first + W1) + KT - 1) / KT : 0;
  if (!SPLIT) return {first, 0, tiles};
  const int half = (tiles + 1) / 2;
  return {first, q == 0 ? 0 : half, q == 0 ? half : tiles};
}

template <int D, bool MASS, bool SPLIT>
__global__ void __launch_bounds__(Geom<D, MASS>::kThreads, 1) prompt_kernel(const __grid_constant__ CUtensorMap mq,
                                                                            const __grid_constant__ CUtensorMap mk,
                                                                            const __grid_constant__ CUtensorMap mv,
                                                                            const __grid_constant__ PromptDev pd) {
  using Geo = Geom<D, MASS>;
  constexpr int QT = Geo::kQT, NS = Geo::kSlots, KT = Geo::kKeys, NU = kUnitSlots;
  constexpr int UQ = SPLIT ? 1 : QT;  // query tiles per unit
  // SPLIT: each stream has half of the K and V slots for its own key tiles, so
  // that neither waits for tiles the other has still to read
  constexpr int KS = SPLIT ? NS / 2 : NS;
  static_assert(!SPLIT || QT == 2, "two streams");
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const PromptArgs& a = pd.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);  // uniform
  const int G = a.cfg.group_size, nh = a.cfg.num_kv_heads;
  const int W1 = pd.tile_tokens;  // query tokens per query tile
  const uint32_t s0 = smem_u32(smem), bars = s0 + Geo::kBar;
  auto bar = [&](int i) { return bars + 8 * i; };
  Shared* sh = reinterpret_cast<Shared*>(smem + Geo::kMisc);
  volatile int* stop = &sh->stop;
  auto ascending = [&] { return a.num_seqs > 32 ? sh->ascending : a.num_seqs; };

  // rows of the Q tiles that no box fills (g not a divisor of 128) stay zero
  if (kRows % G != 0) {
    for (int i = tid; i < QT * Geo::kQTile / 16; i += Geo::kThreads)
      reinterpret_cast<uint4*>(smem + Geo::kQ)[i] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
  }
  if (tid == 0) {
    mbar_init(bar(kBarQFull), 1);
    mbar_init(bar(kBarQEmpty), QT);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarS + i), 1);
      mbar_init(bar(kBarF + i), 4);
      mbar_init(bar(kBarP + i), 4);
      mbar_init(bar(kBarH + i), 4);
      mbar_init(bar(kBarI + i), 4);
      mbar_init(bar(kBarT + i), 4);
      mbar_init(bar(kBarM + i), 4);
      mbar_init(bar(kBarO + i), 1);
      mbar_init(bar(kBarDrain + i), 1);
    }
    for (int i = 0; i < NU; ++i) {
      mbar_init(bar(kBarUFull + i), 1);
      mbar_init(bar(kBarUEmpty + i), 4 * QT + QT + 2);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(bar(kBarKVFull + i), 1);
      mbar_init(bar(kBarKVEmpty + i), UQ);
    }
    mbar_init_fence();
    sh->stop = 0;
    sh->edges = sh->guarded = 0;
    sh->ascending = a.num_seqs;
  }
  if (a.num_seqs > 32) {
    __syncthreads();
    for (int s = tid; s < a.num_seqs; s += Geo::kThreads)
      if (a.cu_seqlens[s + 1] < a.cu_seqlens[s]) atomicMin(&sh->ascending, s);
    __syncthreads();
  }
  if (warp == 0) tmem_alloc512(smem_u32(&sh->tmem));
  // the last warp looks up the first unit meanwhile
  Unit first_unit{0, 0, 0, -1, 0};
  if (warp == 4 * QT + 3) {
    if (lane == 0) {
      tma_prefetch_map(&mq);
      tma_prefetch_map(&mk);
      tma_prefetch_map(&mv);
    }
    if (blockIdx.x < pd.units) first_unit = UnitFinder(pd, ascending(), lane).find(blockIdx.x);
    if (first_unit.n == 0 && a.num_seqs <= kSortedSeqs) first_unit.n = -1;
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = sh->tmem;

  if (warp >= 4 * QT) {
    // (88 and 208 of the 168 registers a thread the block has at launch)
    if constexpr (QT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const int role = warp - 4 * QT;
    if (role < QT) {
      // ------------------------------------------------------------ matrix instructions of query tile `role`
      // The whole warp runs this, on values it knows to be uniform, and one
      // elected lane issues: descriptors then stay in uniform registers (from
      // a single-lane branch each instruction took about 70 cycles to issue).
      const int q = role, base = SPLIT ? q * KS : 0;
      Ring ru, kv{base};
      uint32_t ph_q = 0, ph_f = 0, ph_p = 0;
      int edges = 0;
      bool ok = true;
      const bool leader = elect_one();
      const uint32_t tS = tm + q * Geo::kTile, tP = tS + Geo::kP, tO = tm + Geo::kO + q * D;
      const uint64_t dq = sw128_desc(s0 + Geo::kQ + (SPLIT ? 0 : q) * Geo::kQTile, 0), dk = sw128_desc(s0 + Geo::kKV, 0);
      const uint64_t dv = sw128_desc(s0 + Geo::kKV, KT * 128);
      auto commit = [&](int b) {
        if (leader) mma_commit(bar(b));
      };
      auto wait_kv = [&](const Ring& at) {
        if (!ok) return;
        ok = warp_wait(bar(kBarKVFull + at.slot), at.phase, stop);
        fence_after();
      };
      // S = Q K^T with the K tile at hand
      auto score = [&](const Ring& at) {
        if constexpr (!Geo::kOver) {  // once the softmax has read the last S
          if (!ok || !(ok = warp_wait(bar(kBarF + q), ph_f ^ 1u, stop))) return;
          ph_f ^= 1u;
          fence_after();
        }
        const uint64_t ka = dk + (at.slot * Geo::kSlot >> 4);
        if (leader && ok) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(tS, dq + (((k >> 2) * kRows * 128 + (k & 3) * 32) >> 4),
                   ka + (((k >> 2) * KT * 128 + (k & 3) * 32) >> 4), idesc_m128(KT, false), k != 0);
          mma_commit(bar(kBarS + q));
        }
      };
      // O (+)= P V over the keys [16 k0, 16 k1) of tile j
      auto value = [&](const Ring& at, int j, auto k0, auto k1) {
        const uint64_t va = dv + (at.slot * Geo::kSlot >> 4);
        fence_after();
        if (leader) {
#pragma unroll
          for (int k = decltype(k0)::value; k < decltype(k1)::value; ++k)
            mma_ts(tO, tP + 8 * k, va + (k * 2048 >> 4), idesc_m128(D, true), j > 0 || k > 0);
          if (decltype(k1)::value == KT / 16) mma_commit(bar(kBarO + q));
        }
      };
      constexpr std::integral_constant<int, 0> kBegin{};
      constexpr std::integral_constant<int, KT / 32> kHalf{};
      constexpr std::integral_constant<int, Geo::kOver ? KT * 3 / 64 : 0> kThird{};
      constexpr std::integral_constant<int, KT / 16> kEnd{};
      while (ok) {
        if (!warp_wait(bar(kBarUFull + ru.slot), ru.phase, stop)) break;
        const int n = __shfl_sync(kFull, sh->unit[ru.slot].n, 0);
        const int i0 = __shfl_sync(kFull, sh->unit[ru.slot].run, 0) * W1 * UQ, edge = i0 / KT;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarUEmpty + ru.slot));
        ru.next(NU);
        if (n < 0) break;
        const Work w0 = stream_work<KT, SPLIT>(i0, 0, W1, n), w1 = stream_work<KT, SPLIT>(i0, QT - 1, W1, n);
        const int mine = q == 0 ? w0.count() : w1.count(), steps = max(w0.count(), w1.count());
        if (!(ok = warp_wait(bar(kBarQFull), ph_q, stop))) break;
        ph_q ^= 1u;
        // The ring holds K of step 0, then K of step j + 1 and V of step j for
        // j = 0, 1, ...: of the longer stream, or (SPLIT) of this one
        const int held = SPLIT ? mine : steps;
        auto place = [&] {
          const Ring at = kv;
          kv.next(KS, base);
          return at;
        };
        // the guard's count when V of this stream's step is clean (0: no edge
        // tile); it takes the edge tiles in the order they are loaded
        auto guarded = [&](int step) {
          int until = 0;
          if constexpr (SPLIT) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const Work& y = x == 0 ? w0 : w1;
              if (step < y.count() && y.lo + step >= edge) {
                ++edges;
                if (x == q) until = edges;
              }
            }
          } else if (step >= edge) {
            until = ++edges;
          }
          return until;
        };
        if (held > 0) {
          const Ring k = place();
          wait_kv(k);
          if (mine > 0) score(k);
          commit(kBarKVEmpty + k.slot);
        }
        if (held <= 1) commit(kBarQEmpty);
        for (int j = 0; j < steps && ok; ++j) {
          const int until = guarded(j);
          if (j >= held) continue;
          const bool more = j + 1 < held;
          Ring k = kv;
          if (more) k = place();
          const Ring v = place();
          auto next_scores = [&] {
            if (!more) return;
            wait_kv(k);
            if (j + 1 < mine) score(k);
            commit(kBarKVEmpty + k.slot);
            if (j + 2 == held) commit(kBarQEmpty);
          };
          if constexpr (!Geo::kOver) next_scores();
          wait_kv(v);
          if (!ok) break;
          if (j < mine && !(ok = warp_wait(bar((Geo::kOver ? kBarH : kBarP) + q), ph_p, stop))) break;
          if (until > 0 && !(ok = wait_count(&sh->guarded, until, stop))) break;
          if (j < mine) {
            if constexpr (Geo::kOver) {
              value(v, j, kBegin, kHalf);
              if (!(ok = warp_wait(bar(kBarI + q), ph_p, stop))) break;
              value(v, j, kHalf, kThird);
              if (!(ok = warp_wait(bar(kBarP + q), ph_p, stop))) break;
            }
            value(v, j, kThird, kEnd);
            ph_p ^= 1u;
          }
          commit(kBarKVEmpty + v.slot);
          if constexpr (Geo::kOver) next_scores();
        }
      }
      if (*stop && leader) {  // matrix instructions in flight end before TMEM is freed
        mma_commit(bar(kBarDrain + q));
        const long long t0 = global_ns();
        while (!mbar_try(bar(kBarDrain + q), 0) && global_ns() - t0 < kWaitLimitNs) {
        }
      }
    } else if (role == 2) {
      // ------------------------------------------------------------ loads
      if (lane == 0) {
        Ring ru, ring[2] = {{0}, {SPLIT ? KS : 0}};  // the K and V slots; SPLIT: of each stream
        uint32_t ph_q = 0;
        bool ok = true;
        int issued[2] = {0, 0}, edges = 0;
        while (ok) {
          if (!mbar_wait(bar(kBarUFull + ru.slot), ru.phase, stop)) break;
          const Unit u = sh->unit[ru.slot];
          mbar_arrive(bar(kBarUEmpty + ru.slot));
          ru.next(NU);
          if (u.n < 0) break;
          const int i0 = u.run * W1 * UQ, edge = i0 / KT;
          const Work w0 = stream_work<KT, SPLIT>(i0, 0, W1, u.n), w1 = stream_work<KT, SPLIT>(i0, QT - 1, W1, u.n);
          const int steps = max(w0.count(), w1.count());
          if (!(ok = mbar_wait(bar(kBarQEmpty), ph_q ^ 1u, stop))) break;
          ph_q ^= 1u;
          mbar_expect_tx(bar(kBarQFull), UQ * W1 * G * D * 2);
          for (int q = 0; q < UQ; ++q)
            for (int c = 0; c < D / 64; ++c)
              tma_load(s0 + Geo::kQ + q * Geo::kQTile + c * kRows * 128, &mq, 64 * c, u.head * G,
                       u.first + i0 + q * W1, bar(kBarQFull));
          auto load_tile = [&](const CUtensorMap* map, int j, int x) {
            Ring& kv = ring[x];
            if (!ok || !(ok = mbar_wait(bar(kBarKVEmpty + kv.slot), kv.phase ^ 1u, stop))) return;
            mbar_expect_tx(bar(kBarKVFull + kv.slot), Geo::kSlot);
            for (int c = 0; c < D / 64; ++c)
              tma_load(s0 + Geo::kKV + kv.slot * Geo::kSlot + c * KT * 128, map, 64 * c, u.head, u.first + j * KT,
                       bar(kBarKVFull + kv.slot));
            // the guard may wait for V of an edge tile from now on: the slot's
            // barrier is in this phase until the MMAs have waited for the guard
            if (map == &mv && j >= edge) set_count(&sh->edges, ++edges);
            kv.next(KS, x * KS);
            issued[x] = min(issued[x] + 1, KS);
          };
          auto load = [&](const CUtensorMap* map, int step) {  // in the order the MMA warps take them
            if constexpr (SPLIT) {
              if (step < w0.count()) load_tile(map, w0.lo + step, 0);
              if (step < w1.count()) load_tile(map, w1.lo + step, 1);
            } else if (step < steps) {
              load_tile(map, step, 0);
            }
          };
          load(&mk, 0);
          for (int j = 0; j < steps && ok; ++j) {
            load(&mk, j + 1);
            load(&mv, j);
          }
        }
        if (*stop) {  // copies in flight land before the shared memory is given back
          const long long t0 = global_ns();
          while (issued[0] > 0 && !mbar_try(bar(kBarQFull), ph_q ^ 1u) && global_ns() - t0 < kWaitLimitNs) {
          }
#pragma unroll
          for (int x = 0; x < (SPLIT ? 2 : 1); ++x) {
            Ring& kv = ring[x];
            for (int i = 0; i < issued[x]; ++i) {
              if (kv.slot-- == x * KS) {
                kv.slot = x * KS + KS - 1;
                kv.phase ^= 1u;
              }
              while (!mbar_try(bar(kBarKVFull + kv.slot), kv.phase) && global_ns() - t0 < kWaitLimitNs) {
              }
            }
          }
        }
      }
    } else if (role == 3) {
      // ------------------------------------------------------------ units, and the V guard
      if (blockIdx.x == 0) {
        for (int s = lane; s < a.num_seqs; s += 32) {
          if (!seq_ok(a.cu_seqlens[s], a.cu_seqlens[s + 1], a.total_tokens, a.max_seq_tokens))
            report_error(a.dev_status, KVQ_ERR_DEVICE_BOUNDS);
        }
      }
      // Units of this CTA: every gridDim.x-th, in alternating direction (with
      // units longest first the CTAs end up with about the same work).
      Ring pub, ru, ring[2] = {{0}, {SPLIT ? KS : 0}};
      const UnitFinder finder(pd, ascending(), lane);
      int round = 1;
      bool more = true;
      auto publish = [&](Unit u) {  // the next unit from u on, n = -1 after the last
        while (u.n == 0) {
          const long long x = static_cast<long long>(round) * gridDim.x +
                              ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
          ++round;
          if (x < pd.units) u = finder.find(static_cast<int>(x));
          if (x >= pd.units || (u.n == 0 && a.num_seqs <= kSortedSeqs)) u.n = -1;
        }
        more = u.n > 0;
        if (!warp_wait(bar(kBarUEmpty + pub.slot), pub.phase ^ 1u, stop)) return;
        if (lane == 0) {
          sh->unit[pub.slot] = u;
          sh->odd_v[pub.slot] = 0;
          mbar_arrive(bar(kBarUFull + pub.slot));
        }
        pub.next(NU);
      };
      const Unit unknown{0, 0, 0, 0, 0};
      publish(first_unit);
      if (more) publish(unknown);
      int edges = 0;
      while (warp_wait(bar(kBarUFull + ru.slot), ru.phase, stop)) {
        const Unit u = sh->unit[ru.slot];
        const int uslot = ru.slot;
        ru.next(NU);
        if (u.n < 0) break;
        // V of the tiles that hold keys some row does not see: rows past the
        // sequence and values that are not finite become zero
        const int i0 = u.run * W1 * UQ, edge = i0 / KT;
        const Work w0 = stream_work<KT, SPLIT>(i0, 0, W1, u.n), w1 = stream_work<KT, SPLIT>(i0, QT - 1, W1, u.n);
        const int steps = max(w0.count(), w1.count());
        auto holds = [&](int step, int x) { return step < (SPLIT ? (x == 0 ? w0 : w1).count() : steps); };
        bool ok = true;
        for (int step = -1; step < steps && ok; ++step) {
#pragma unroll
          for (int x = 0; x < (SPLIT ? 2 : 1); ++x) {
            Ring& kv = ring[x];
            if (holds(step + 1, x)) kv.next(KS, x * KS);  // K of step + 1
            if (step < 0 || !holds(step, x) || !ok) continue;
            const int j = (SPLIT && x == 1 ? w1.lo : 0) + step;
            if (j < edge) {
              kv.next(KS, x * KS);
              continue;
            }
            ++edges;
            if (!(ok = wait_count(&sh->edges, edges, stop))) continue;
            if (!(ok = warp_wait(bar(kBarKVFull + kv.slot), kv.phase, stop))) continue;
            uint4* p = reinterpret_cast<uint4*>(smem + Geo::kKV + kv.slot * Geo::kSlot);
            const int held = min(KT, u.n - j * KT);  // rows of the sequence
            if (held < KT)
              for (int c = 0; c < D / 64; ++c)  // (64 channels of a row are 8 x 16 bytes)
                for (int i = held * 8 + lane; i < KT * 8; i += 32) p[c * KT * 8 + i] = make_uint4(0, 0, 0, 0);
            __syncwarp();
            // x * 0 is NaN just where x is not finite
            const __half2 zero = __float2half2_rn(0.f);
            __half2 probe[4] = {zero, zero, zero, zero};
#pragma unroll 8
            for (int i = lane; i < Geo::kSlot / 16; i += 32) {
              const uint4 x = p[i];
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) probe[e] = __hfma2(u32_as_h2(w[e]), zero, probe[e]);
            }
            const __half2 all = __hadd2(__hadd2(probe[0], probe[1]), __hadd2(probe[2], probe[3]));
            const bool odd = __any_sync(kFull, __hisnan(__low2half(all)) || __hisnan(__high2half(all)));
            if (odd) {
              for (int i = lane; i < Geo::kSlot / 16; i += 32) {
                uint4 x = p[i];
                uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if ((w[e] & 0x7C00u) == 0x7C00u) w[e] &= 0xFFFF0000u;
                  if ((w[e] & 0x7C000000u) == 0x7C000000u) w[e] &= 0x0000FFFFu;
                }
                p[i] = x;
              }
            }
            if (odd) sh->odd_v[uslot] = 1;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) set_count(&sh->guarded, edges);
            kv.next(KS, x * KS);
          }
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(bar(kBarUEmpty + uslot));
        if (more) publish(unknown);
      }
    }
  } else {
    // -------------------------------------------------------------- softmax
    if constexpr (QT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int q = warp >> 2, row = tid & 127;
    const uint32_t tlane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tm + q * Geo::kTile + tlane, tP = tS + Geo::kP, tO = tm + Geo::kO + q * D + tlane;
    const int T = a.cfg.tile_tokens, wid = min(T, KT), ent = KT / wid;  // keys per mass entry, entries per tile
    float* s_m = reinterpret_cast<float*>(smem + Geo::kStat) + q * 2 * kRows;
    float* s_w = s_m + kRows;
    // token of this row in the query tile, its row in the output from the
    // tile's first; the same of the piece this lane writes in store k below
    const int row_token = row / G, own = row_token * nh * G + row % G;
    int put_token[4], put[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = (warp & 3) * 32 + 8 * k + (lane >> 2);
      put_token[k] = r < W1 * G ? r / G : 1 << 24;  // (no token)
      put[k] = ((r / G) * nh * G + r % G) * D + 8 * (lane & 3);
    }
    Ring ru;
    uint32_t ph_m = 0;
    uint32_t ph_s = 0, ph_o = 0, ph_t = q == 0 ? 1u : 0u;  // (query tile 0 has the first turn)
    const bool leader = elect_one();
    auto publish = [&](int b) {  // this warp's TMEM accesses so far
      fence_before();
      __syncwarp();
      mbar_arrive_if(leader, bar(b + q));
    };
    while (warp_wait(bar(kBarUFull + ru.slot), ru.phase, stop)) {
      const Unit u = sh->unit[ru.slot];
      const int uslot = ru.slot;
      ru.next(NU);
      if (u.n < 0) break;
      const Work w = stream_work<KT, SPLIT>(u.run * W1 * UQ, q, W1, u.n);
      const int first = w.first, nk = w.count();         // the query tile's first token; this stream's key tiles
      const int ti = first + row_token;                  // this row's token
      const bool live = row < W1 * G && ti < u.n;
      const int vis = live ? ti : u.n - 1;               // last key this row sees
      const int masked = first / KT;                     // tiles from here on need the mask
      const long long slot = MASS && nk > 0 ? mass_slot(pd, u, u.run * UQ + (SPLIT ? 0 : q)) : -1;
      float* scr = pd.scratch + (static_cast<size_t>(blockIdx.x) * QT + (SPLIT ? 0 : q)) * pd.max_tiles_k * (ent + 1) * kRows + row;
      // tiles that both streams have: they take turns
      const int turns = !Geo::kTurns ? 0 : min(nk, stream_work<KT, SPLIT>(u.run * W1 * UQ, 1 - q, W1, u.n).count());
      float m = -INFINITY, l = 0.f;
      const float spare = spare_bits(min(u.n, first + W1));
      bool ok = true;
      for (int step = 0; step < nk; ++step) {
        const int j = w.lo + step;  // key tile
        if (!(ok = warp_wait(bar(kBarS + q), ph_s, stop))) break;
        ph_s ^= 1u;
        fence_after();
        float s[KT];
        // mask of the keys [o, e) and their maximum (times the scale)
        auto top_of = [&](auto from, auto to) {
          constexpr int o = decltype(from)::value, e = decltype(to)::value;
          if (j >= masked) {
            const int lim = vis - j * KT;  // last key of the tile that the row sees
#pragma unroll
            for (int c = o; c < e; ++c) s[c] = c <= lim ? s[c] : -INFINITY;
          }
          float mx[4] = {s[o], s[o + 1], s[o + 2], s[o + 3]};
#pragma unroll
          for (int c = o + 4; c < e - 4; c += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = max3nan(mx[k], s[c + k], s[c + 4 + k]);
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = max3nan(mx[k], s[e - 4 + k], s[e - 4 + k]);
          // (rounded as it is kept, not again inside a multiply-add)
          const float t = __fmul_rn(max3nan(mx[0], mx[1], max3nan(mx[2], mx[3], mx[3])), pd.qscale);
          if (!(t < kFar)) l = NAN;  // a NaN or a score of +inf: the row is NaN (-inf has no weight)
          return t;
        };
        // The maximum moves to `top` in the lanes where it is more than kLazy
        // larger (m = -inf before the first finite score); O and l follow.
        auto grow = [&](float top) {
          float alpha = 1.f;
          if (top > m + kLazy && top > -kFar) {
            const float to = top - spare;
            alpha = ex2(m - to);
            m = to;
            l *= alpha;
          }
          if (step == 0) return;
          // the last P V is done (with P over S this tile's score MMA came after it)
          if (!Geo::kOver && !(ok = warp_wait(bar(kBarO + q), ph_o ^ 1u, stop))) return;
          fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 8) {  // few registers: the scores stay in theirs
            float o[8];
            tmem_ld8(tO + c, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= alpha;
            tmem_st8(tO + c, o);
          }
        };
        float2 part[KT / 32];  // sums of 32 keys
        // weights of the keys [o, e) into p
        auto weigh = [&](auto from, auto to, uint32_t* p) {
          constexpr int o = decltype(from)::value, e = decltype(to)::value;
          const float mu = m == -INFINITY ? 0.f : m;  // a row with no finite score so far
          const float2 sc2 = make_float2(pd.qscale, pd.qscale), mu2 = make_float2(-mu, -mu);
#pragma unroll
          for (int c = o; c < e; c += 2) {
            const float2 x = __ffma2_rn(make_float2(s[c], s[c + 1]), sc2, mu2);
            const float2 y = make_float2(ex2(x.x), ex2(x.y));
            float2& sum = part[c / 32];
            sum = c % 32 == 0 ? y : __fadd2_rn(sum, y);
            p[(c - o) / 2] = h2_as_u32(__float22half2_rn(y));
          }
        };
        auto take_turn = [&] {
          if (Geo::kTurns && step < turns && ok) {
            ok = warp_wait(bar(kBarT + q), ph_t, stop);
            ph_t ^= 1u;
          }
        };
        auto pass_turn = [&] {
          if (Geo::kTurns && step < turns) mbar_arrive_if(leader, bar(kBarT + 1 - q));
        };
        constexpr std::integral_constant<int, 0> k0{};
        constexpr std::integral_constant<int, 32> k32{};
        constexpr std::integral_constant<int, 64> k64{};
        constexpr std::integral_constant<int, KT - 32> k96{};
        constexpr std::integral_constant<int, KT> kEnd{};
        if constexpr (Geo::kOver) {
          // The tile goes in runs of keys.  The first 32 keys' weights are
          // taken relative to the maximum up to them while the other scores
          // are still on their way and being compared; P V starts on 64 and
          // then 96 keys while the weights of the rest are computed, and the
          // other query tile takes its turn before the last 16.  Each part of
          // P is waited for and published a run later than it is stored.
          uint32_t pa[KT / 4], pb[KT / 8];
          constexpr std::integral_constant<int, KT - 16> k112{};
          tmem_ld32<0>(tS, s);
          tmem_wait32<0>(s);
          tmem_ld32<32>(tS + 32, s);
          tmem_ld32<KT - 64>(tS + KT - 64, s);
          tmem_ld32<KT - 32>(tS + KT - 32, s);
          float top = top_of(k0, k32);
          if (__any_sync(kFull, top > m + kLazy)) grow(top);
          take_turn();
          weigh(k0, k32, pa);
          tmem_wait32<32>(s);
          tmem_wait32<KT - 64>(s);
          tmem_wait32<KT - 32>(s);
          top = top_of(k32, kEnd);
          if (__any_sync(kFull, top > m + kLazy)) {  // rare: the first run again
            grow(top);
            weigh(k0, k32, pa);
          }
          if (!ok) break;
          weigh(k32, k64, pa + 16);
          tmem_st32<0>(tP, pa);  // over 32 columns of scores already read
          weigh(k64, k96, pb);
          tmem_wait_st();
          publish(kBarH);
          tmem_st16(tP + KT / 4, pb);
          weigh(k96, k112, pa);
          pass_turn();
          tmem_wait_st();
          publish(kBarI);
          weigh(k112, kEnd, pa + 8);
          tmem_st16(tP + KT / 2 - 16, *reinterpret_cast<uint32_t(*)[KT / 8]>(pa));
        } else {
          uint32_t p[KT / 2];
          tmem_ld32<0>(tS, s);
          tmem_ld32<32>(tS + 32, s);
          if constexpr (KT == 128) {
            tmem_ld32<KT - 64>(tS + KT - 64, s);
            tmem_ld32<KT - 32>(tS + KT - 32, s);
          }
          tmem_wait32<0>(s);
          tmem_wait32<32>(s);
          if constexpr (KT == 128) {
            tmem_wait32<KT - 64>(s);
            tmem_wait32<KT - 32>(s);
          }
          publish(kBarF);  // the next scores may come
          const float top = top_of(k0, kEnd);
          if (__any_sync(kFull, top > m + kLazy)) grow(top);
          take_turn();
          weigh(k0, kEnd, p);
          pass_turn();
          // the last P V is done: P may be written
          if (step > 0 && ok) ok = warp_wait(bar(kBarO + q), ph_o ^ 1u, stop);
          if (!ok) break;
          fence_after();
          tmem_st32<0>(tP, p);
          if constexpr (KT == 128) tmem_st32<KT / 2 - 32>(tP + 32, p);
        }
        tmem_wait_st();
        publish(kBarP);
        const float mu = m == -INFINITY ? 0.f : m;
        ph_o ^= 1u;
        float ps[KT / 32];
        float all = 0.f;
#pragma unroll
        for (int k = 0; k < KT / 32; ++k) all += ps[k] = part[k].x + part[k].y;
        l += all;
        if constexpr (MASS) {
          if (slot >= 0) {
            float* d = scr + static_cast<size_t>(j) * (ent + 1) * kRows;
            if (wid == 32) {
#pragma unroll
              for (int k = 0; k < KT / 32; ++k) d[k * kRows] = ps[k];
            } else if (wid == 64) {
#pragma unroll
              for (int k = 0; k < KT / 64; ++k) d[k * kRows] = ps[2 * k] + ps[2 * k + 1];
            } else {
              d[0] = all;
            }
            d[ent * kRows] = mu;
          }
        }
      }
      if (!ok) break;
      float part0 = 1.f, part1 = 0.f;  // SPLIT: the streams' shares of the merged row
      bool other = false;              // stream 1 has some
      if constexpr (SPLIT) {
        float* s_m1 = reinterpret_cast<float*>(smem + Geo::kStat) + 2 * kRows;  // stream 1's m and l
        float* s_l1 = s_m1 + kRows;
        if (q == 1) {
          if (nk > 0) {
            if (!warp_wait(bar(kBarO + 1), ph_o ^ 1u, stop)) break;
            s_m1[row] = m;
            s_l1[row] = l;
          }
          __threadfence_block();
          publish(kBarM);
          if (!warp_wait(bar(kBarM), ph_m, stop)) break;  // merged: O and the scratch are free again
          ph_m ^= 1u;
        } else {
          other = stream_work<KT, SPLIT>(u.run * W1 * UQ, 1, W1, u.n).count() > 0;
          if (!warp_wait(bar(kBarM + 1), ph_m, stop)) break;
          ph_m ^= 1u;
          if (other) {  // the log-sum-exp merge of the two
            const float m1 = s_m1[row], top = fmaxf(m, m1);
            part0 = m == -INFINITY ? 0.f : ex2(m - top);
            part1 = m1 == -INFINITY ? 0.f : ex2(m1 - top);
            l = l * part0 + s_l1[row] * part1;
            m = top;
          }
        }
      }
      if (nk > 0 && (!SPLIT || q == 0)) {
        // ---- the tile's rows
        if (!warp_wait(bar(kBarO + q), ph_o ^ 1u, stop)) break;
        fence_after();
        const bool odd = *static_cast<volatile int*>(&sh->odd_v[uslot]) != 0;
        const float inv = 1.f / l;
        const size_t base = static_cast<size_t>(u.first + first) * nh * G + u.head * G;  // row 0 of the tile
        // 32 channels of the warp's 32 rows at a time through shared memory, so
        // that a store writes 64 bytes of each of eight rows (16 bytes of each
        // of 32 rows took 2200 to 4300 cycles a tile); 16-byte pieces of a row
        // are exchanged so that neither side meets bank conflicts
        unsigned char* stage = smem + Geo::kStage + warp * 2048;
        __half* out = static_cast<__half*>(a.out) + base * D;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 64) {
          float o[64];
          tmem_ld32<0>(tO + c0, o);
          tmem_ld32<32>(tO + c0 + 32, o);
          tmem_wait32<0>(o);
          tmem_wait32<32>(o);
          if constexpr (SPLIT) {
            if (other) {
#pragma unroll
              for (int c = 0; c < 64; c += 8) {
                float x[8];
                tmem_ld8(tO + D + c0 + c, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[c + e] = o[c + e] * part0 + x[e] * part1;
              }
            }
          }
          // A mean of finite values is at most the largest of them; the weights'
          // rounding can take it past that by 2^-11 of it, and past fp16's
          // largest: then 2^-11 less for these channels of the row.  (A search
          // for such values alone, mended one by one behind a branch, took 4%
          // of a short prompt's time, this takes 1.5%.)
          float big = 0.f;
#pragma unroll
          for (int e = 0; e < 64; e += 2) big = max3abs(big, o[e], o[e + 1]);
          big *= inv;
          const float mean = big > 65504.f && big < 66000.f ? inv * (1.f - 0x1p-11f) : inv;
#pragma unroll
          for (int e = 0; e < 64; ++e) o[e] *= mean;
          if (odd && live) {  // the values the V guard left out, to the rows that see them
            for (int key = u.run * W1 * UQ / KT * KT; key <= vis; ++key) {
              const __half* vr = static_cast<const __half*>(a.v) + static_cast<size_t>(u.first + key) * a.v_stride +
                                 u.head * D + c0;
#pragma unroll
              for (int e = 0; e < 64; ++e) {
                const float x = __half2float(vr[e]);
                if (!(fabsf(x) <= 65504.f)) o[e] += x;
              }
            }
          }
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float* x = o + c + 8 * e;
              uint4 w;
              w.x = h2_as_u32(__floats2half2_rn(x[0], x[1]));
              w.y = h2_as_u32(__floats2half2_rn(x[2], x[3]));
              w.z = h2_as_u32(__floats2half2_rn(x[4], x[5]));
              w.w = h2_as_u32(__floats2half2_rn(x[6], x[7]));
              *reinterpret_cast<uint4*>(stage + lane * 64 + ((e ^ (lane >> 1)) & 3) * 16) = w;
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = 8 * k + (lane >> 2);
              const uint4 w = *reinterpret_cast<const uint4*>(stage + r * 64 + ((lane ^ (r >> 1)) & 3) * 16);
              if (first + put_token[k] < u.n) *reinterpret_cast<uint4*>(out + put[k] + c0 + c) = w;
            }
            __syncwarp();
          }
        }
        if (live && a.lse != nullptr) a.lse[base + own] = (m + log2f(l)) * 0.6931471805599453f;
        if (MASS && slot >= 0) {
          const bool counts = live && (a.mass_window == 0 || ti >= u.n - a.mass_window);
          s_m[row] = m == -INFINITY ? 0.f : m;
          s_w[row] = counts ? inv : 0.f;
          asm volatile("bar.sync %0, 128;" ::"r"(1 + q) : "memory");
          float* dst = pd.part + static_cast<size_t>(slot) * pd.max_tiles_k * ent;
          const float* base = scr - row;
          // a warp an entry, four rows a lane (whole lines: with the entries
          // across the lanes this took 3.8 us a unit), then the lanes by butterfly
          const float4 f = *reinterpret_cast<const float4*>(s_m + 4 * lane);
          const float4 w = *reinterpret_cast<const float4*>(s_w + 4 * lane);
          // A row that does not count has weight 0, and its sums may be
          // anything.  An entry that a row does not see is none of its
          // weight, whatever the row is.  A share without a finite score is
          // relative to 0 and not to a maximum, which may lie above f.
          int sees[4];  // tokens of this lane's rows
#pragma unroll
          for (int r = 0; r < 4; ++r) sees[r] = first + (4 * lane + r) / G;
          auto term = [](float x, float y, float f, float w, bool seen) {
            return w != 0.f && seen ? x * ex2(fminf(y - f, 0.f)) * w : 0.f;
          };
          const int stride = (ent + 1) * kRows, ent_bits = ent == 4 ? 2 : ent - 1;
          const int entries = (SPLIT ? (min(u.n, first + W1) + KT - 1) / KT : nk) * ent;
#pragma unroll 4
          for (int i = warp & 3; i < entries; i += 4) {
            const float* tile = base + static_cast<size_t>(i >> ent_bits) * stride + 4 * lane;
            const float4 x = *reinterpret_cast<const float4*>(tile + (i & (ent - 1)) * kRows);
            const float4 y = *reinterpret_cast<const float4*>(tile + ent * kRows);
            const int key = i * wid;  // the entry's first
            const float sum =
                warp_sum((term(x.x, y.x, f.x, w.x, sees[0] >= key) + term(x.y, y.y, f.y, w.y, sees[1] >= key)) +
                         (term(x.z, y.z, f.z, w.z, sees[2] >= key) + term(x.w, y.w, f.w, w.w, sees[3] >= key)));
            if (lane == 0) dst[i] = sum;
          }
          asm volatile("bar.sync %0, 128;" ::"r"(1 + q) : "memory");
        }
        fence_before();
      }
      if constexpr (SPLIT) {
        if (q == 0) publish(kBarM);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarUEmpty + uslot));
    }
    if (*stop && tid == 0) report_error(a.dev_status, KVQ_ERR_DEVICE_TIMEOUT);
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 0) tmem_free512(tm);
}

// mass[s][t] += the partial masses of the query tiles of sequence s that reach
// tile t.  A CTA per 32 entries (min(T, KT) keys each): lanes over the
// entries, warps over the (run, head) rows with a fixed stride, then the warps
// in order.  The rows of a sequence lie one after another (mass_slot).
constexpr int kMassWarps = 32;
__global__ void __launch_bounds__(kMassWarps * 32) prompt_mass_kernel(PromptDev pd, int KT) {
  __shared__ float s_sum[kMassWarps][33];
  const PromptArgs& a = pd.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int T = a.cfg.tile_tokens, W1 = pd.tile_tokens, nh = a.cfg.num_kv_heads;
  const int wid = min(T, KT), per = T / wid;  // keys per entry, entries per tile of T (1 or 2)
  const int e = blockIdx.x * 32 + lane;
  Unit u{static_cast<int>(blockIdx.y), 0, 0, 0, 0};
  u.n = seq_len(a, u.seq, u.first);
  bool down = false;  // behind a descent of the prefix sums
  if (u.seq > 0) {
    for (int s = threadIdx.x; s < u.seq; s += kMassWarps * 32) down |= a.cu_seqlens[s + 1] < a.cu_seqlens[s];
    down = __syncthreads_or(down);
  }
  cudaGridDependencySynchronize();
  if (down || blockIdx.x * 32 * wid >= u.n) return;
  const int w0 = a.mass_window == 0 ? 0 : max(0, u.n - a.mass_window) / W1;
  const int rows = ((u.n + W1 - 1) / W1 - w0) * nh;  // from query tile w0 on
  // the first row that sees the entry (rows before it may not have written it)
  const int from = e * wid < u.n ? max(0, e * wid / W1 - w0) * nh : rows;
  const size_t stride = static_cast<size_t>(pd.max_tiles_k) * (KT / wid);
  const float* p = pd.part + static_cast<size_t>(mass_slot(pd, u, w0)) * stride + e;
  float sum = 0.f;
#pragma unroll 8
  for (int x = warp; x < rows; x += kMassWarps)
    if (x >= from) sum += p[x * stride];
  s_sum[warp][lane] = sum;
  __syncthreads();
  if (warp != 0) return;
  sum = 0.f;
  for (int w = 0; w < kMassWarps; ++w) sum += s_sum[w][lane];
  if (per == 2) sum += __shfl_down_sync(kFull, sum, 1);
  const int t = e / per;
  if (e % per == 0 && e * wid < u.n && t < a.max_tiles) a.mass[static_cast<size_t>(u.seq) * a.max_tiles + t] += sum;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
  }();
  return fn;
}

// rows [tokens][heads][d] fp16, `stride` elements from row to row: boxes of 64
// channels x box_heads x box_rows, 128-byte swizzle, zeros past the last row
bool make_map(CUtensorMap* m, const void* base, int d, int heads, int tokens, long long stride, int box_heads,
              int box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(stride) * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int tile_tokens(const kvq_config& cfg) { return kRows / cfg.group_size; }
int query_tiles(const kvq_config& cfg) { return cfg.head_dim == 256 ? Geom<256, true>::kQT : Geom<128, true>::kQT; }
// keys per tile of a call with masses
int mass_keys(const kvq_config& cfg) {
  switch (cfg.head_dim) {
    case 64: return Geom<64, true>::kKeys;
    case 128: return Geom<128, true>::kKeys;
    default: return Geom<256, true>::kKeys;
  }
}

struct PromptSizes {
  long long units;
  bool split;  // a unit is one query tile, its key tiles shared out over two streams
  int max_tiles_k, window_runs, grid;
  size_t scratch_floats, part_floats;
};
PromptSizes prompt_sizes(const kvq_config& cfg, int num_seqs, int total_tokens, int max_seq_tokens, int window,
                         int sms) {
  PromptSizes z;
  const int W1 = tile_tokens(cfg), keys = mass_keys(cfg), ent = keys / std::min(keys, cfg.tile_tokens);
  z.units = prompt_units(cfg, num_seqs, total_tokens);
  // With no more units than SMs a call takes as long as its longest unit: then
  // a unit is one query tile and the CTA's two streams take half of its keys
  // each.  Pairs of query tiles against halves of the keys, us in a graph, d =
  // 128 / d = 64: 34 units of pairs (1024 tokens, 8 heads over 2) 21.5 against
  // 16.1 / 20.1 against 14.3; 148 (3050, 12 over 4) 49.5, 37.7 / 44.7, 32.1, with
  // masses 59.7, 47.4 / 56.7, 41.6.  Beyond, CTAs take several units and a pair
  // loads each key tile once for two: 192 (4000, 12 over 4) 64.3, 63.6 / 57.2,
  // 52.1; 256 (4096, 16 over 2) 80, 95 / 71, 76.
  z.split = query_tiles(cfg) == 2 && z.units <= sms;
  if (z.split) z.units = (static_cast<long long>(total_tokens) / W1 + num_seqs) * cfg.num_kv_heads;
  z.max_tiles_k = (max_seq_tokens + keys - 1) / keys;
  z.window_runs = window == 0 ? 0 : std::min((window - 1) / W1 + 2, (max_seq_tokens + W1 - 1) / W1);
  z.grid = static_cast<int>(std::min<long long>(z.units, sms));
  z.scratch_floats = static_cast<size_t>(z.grid) * query_tiles(cfg) * z.max_tiles_k * (ent + 1) * kRows;
  const size_t runs = window == 0 ? static_cast<size_t>(total_tokens) / W1 + num_seqs
                                  : static_cast<size_t>(num_seqs) * z.window_runs;
  z.part_floats = runs * cfg.num_kv_heads * z.max_tiles_k * ent;
  return z;
}

template <int D, bool MASS, bool SPLIT>
cudaError_t launch_prompt_kernel(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                                 const PromptDev& pd, int grid, cudaStream_t s) {
  using Geo = Geom<D, MASS>;
  static PerContext<int> opted_in;  // to the shared memory
  auto kern = prompt_kernel<D, MASS, SPLIT>;
  int done = 0;
  const cudaError_t e = opted_in.get(&done, [&](int* v) {
    *v = 1;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo::kSmem);
  });
  if (e != cudaSuccess) return e;
  kern<<<grid, Geo::kThreads, Geo::kSmem, s>>>(mq, mk, mv, pd);
  return cudaGetLastError();
}

template <int D, bool MASS>
cudaError_t launch_prompt(const PromptArgs& a, cudaStream_t s) {
  using Geo = Geom<D, MASS>;
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const PromptSizes z = prompt_sizes(a.cfg, a.num_seqs, a.total_tokens, a.max_seq_tokens, a.mass_window, sms);
  const int G = a.cfg.group_size, nh = a.cfg.num_kv_heads;
  CUtensorMap mq, mk, mv;
  if (!make_map(&mq, a.q, D, nh * G, a.total_tokens, a.q_stride, G, kRows / G) ||
      !make_map(&mk, a.k, D, nh, a.total_tokens, a.k_stride, 1, Geo::kKeys) ||
      !make_map(&mv, a.v, D, nh, a.total_tokens, a.v_stride, 1, Geo::kKeys))
    return cudaErrorInvalidValue;
  PromptDev pd{};
  pd.a = a;
  pd.tile_tokens = tile_tokens(a.cfg);
  pd.unit_tokens = pd.tile_tokens * (z.split ? 1 : Geo::kQT);  // 16 .. 256
  pd.unit_magic = static_cast<uint32_t>((1ull << 32) / pd.unit_tokens) + 1;
  pd.units = static_cast<int>(z.units);
  pd.max_tiles_k = z.max_tiles_k;
  pd.window_runs = z.window_runs;
  pd.qscale = a.softmax_scale * kLog2e;
  pd.scratch = static_cast<float*>(a.workspace);
  pd.part = pd.scratch + z.scratch_floats;
  if constexpr (Geo::kQT == 2)
    e = z.split ? launch_prompt_kernel<D, MASS, true>(mq, mk, mv, pd, z.grid, s)
                : launch_prompt_kernel<D, MASS, false>(mq, mk, mv, pd, z.grid, s);
  else
    e = launch_prompt_kernel<D, MASS, false>(mq, mk, mv, pd, z.grid, s);
  if (e != cudaSuccess || !MASS) return e;
  const int wid = std::min(a.cfg.tile_tokens, Geo::kKeys);
  return launch_behind(prompt_mass_kernel, dim3((a.max_seq_tokens + 32 * wid - 1) / (32 * wid), a.num_seqs),
                       kMassWarps * 32, s, pd, static_cast<int>(Geo::kKeys));
}

// ------------------------------------------------------------------ self-test
// This file's bounded wait on a barrier that nothing arrives at.
__global__ void selftest_wait_prompt_kernel(int32_t* dev_status) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int stop;
  stop = 0;
  mbar_init(smem_u32(&bar), 1);
  mbar_init_fence();
  if (!mbar_wait(smem_u32(&bar), 0, &stop)) report_error(dev_status, KVQ_ERR_DEVICE_TIMEOUT);
}

}  // namespace

cudaError_t launch_selftest_wait_prompt(int32_t* dev_status, cudaStream_t s) {
  selftest_wait_prompt_kernel<<<1, 1, 0, s>>>(dev_status);
  return cudaGetLastError();
}

long long prompt_units(const kvq_config& cfg, int num_seqs, int total_tokens) {
  return (static_cast<long long>(total_tokens) / (tile_tokens(cfg) * query_tiles(cfg)) + num_seqs) * cfg.num_kv_heads;
}

size_t prompt_workspace_bytes(const kvq_config& cfg, int num_seqs, int total_tokens, int max_seq_tokens, int window,
                              int sms) {
  const PromptSizes z = prompt_sizes(cfg, num_seqs, total_tokens, max_seq_tokens, window, sms);
  return (z.scratch_floats + z.part_floats) * sizeof(float);
}

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t s) {
  const bool mass = a.mass != nullptr;
  switch (a.cfg.head_dim) {
    case 64: return mass ? launch_prompt<64, true>(a, s) : launch_prompt<64, false>(a, s);
    case 128: return mass ? launch_prompt<128, true>(a, s) : launch_prompt<128, false>(a, s);
    default: return mass ? launch_prompt<256, true>(a, s) : launch_prompt<256, false>(a, s);
  }
}

}  // namespace kvq
