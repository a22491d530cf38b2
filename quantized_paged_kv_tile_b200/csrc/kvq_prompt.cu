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
// A work unit is (sequence, run of kUnitTokens query tokens, KV head): its
// 128 rows are tokens x the g query heads of the KV head, token-major, one
// row per TMEM lane.  Per tile of 128 keys: S = Q K^T (tcgen05, fp32 in
// TMEM), the softmax of a row in one thread, P as fp16 over S in TMEM, and
// O += P V with V read as it lies in memory (keys as rows: an MN-major B
// operand).  P is rounded to fp16 (half a step is 2^-11 of each weight; the
// sum l takes the unrounded weights), everything else stays in fp32.
//
// What a mask hides never reaches a result: masked scores become -inf by
// selection; V rows past the sequence are zeroed in shared memory; V values
// of the tiles that straddle the diagonal that are not finite are replaced
// by zero there and added, unweighted, to exactly the rows that see them.
//
// Mass (optional): per row and run of T keys the sum of the weights, with the
// maximum it is relative to, goes to a scratch area of the CTA; once a unit's
// l and m are final, the rows that count are weighted and summed, and a second
// kernel adds the units of a sequence to its masses in a fixed order.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kvq_device.cuh"
#include "kvq_sm100.cuh"

namespace kvq {

namespace {

using namespace sm100;

constexpr int kRows = 128;    // query rows per query tile (TMEM lanes)
// The running maximum a row's weights are relative to follows the true one
// only once that is more than 2^kLazy larger: weights reach 2^8 then (fp16 and
// the fp32 sums hold that as exactly as 1), and O is rescaled rarely.
constexpr float kLazy = 8.f;
// up to this many sequences the units are taken longest first
constexpr int kSortedSeqs = 1024;

struct PromptDev {
  PromptArgs a;
  int tile_tokens;     // query tokens per query tile
  int unit_tokens;     // query tokens per unit (one or two query tiles)
  int units;           // host bound on the number of units
  int max_tiles_k;     // key tiles of the longest sequence
  int window_runs;     // query tiles per (sequence, head) that can hold counted queries; 0: all
  float qscale;        // softmax_scale * log2 e
  float* scratch;      // per CTA and query tile [max_tiles_k][entries per key tile + 1][kRows]
  float* part;         // per query tile of the call [max_tiles_k * entries per key tile]
};

// Length and first row of sequence s; 0 tokens if the prefix sums are bad.
__device__ __forceinline__ int seq_len(const PromptArgs& a, int s, int& first) {
  first = a.cu_seqlens[s];
  const int end = a.cu_seqlens[s + 1];
  const bool ok = first >= 0 && end >= first && end <= a.total_tokens && end - first <= a.max_seq_tokens;
  return ok ? end - first : 0;
}

struct Unit {
  int seq, run, head, n, first;  // n = 0: nothing here
};

// Where unit u sits; the whole warp calls it.  Up to kSortedSeqs sequences:
// units in descending order of their run index (so of their keys), from a
// binary search over the levels, count(c) = number of units of run >= c.
// More: sequence s owns the slots from first_s / W + s on, found by binary
// search; slots past its units are empty.
__device__ Unit locate_unit(const PromptDev& pd, int u, int lane) {
  const PromptArgs& a = pd.a;
  const int nh = a.cfg.num_kv_heads, W = pd.unit_tokens, B = a.num_seqs;
  Unit r{0, 0, u % nh, 0, 0};
  const int x = u / nh;
  if (B <= kSortedSeqs) {
    auto count = [&](int c) {
      int k = 0, f;
      for (int s = lane; s < B; s += 32) k += max(0, (seq_len(a, s, f) + W - 1) / W - c);
      return __reduce_add_sync(kFull, k);
    };
    if (count(0) <= x) return r;
    int lo = 0, hi = (a.max_seq_tokens + W - 1) / W, above = 0;
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
    for (int s0 = 0; s0 < B; s0 += 32) {
      const int s = s0 + lane;
      int f = 0;
      const int n = s < B ? seq_len(a, s, f) : 0;
      const unsigned has = __ballot_sync(kFull, (n + W - 1) / W > lo);
      if (k < __popc(has)) {
        const int src = __fns(has, 0, k + 1);
        r.seq = s0 + src;
        r.run = lo;
        r.n = __shfl_sync(kFull, n, src);
        r.first = __shfl_sync(kFull, f, src);
        return r;
      }
      k -= __popc(has);
    }
    return r;
  }
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (max(a.cu_seqlens[mid], 0) / W + mid <= x) lo = mid; else hi = mid;
  }
  int f = 0;
  const int n = seq_len(a, lo, f);
  r.run = x - (f / W + lo);
  if (r.run >= 0 && r.run < (n + W - 1) / W) {
    r.seq = lo;
    r.n = n;
    r.first = f;
  }
  return r;
}

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

__device__ __forceinline__ float max3f(float x, float y, float z) { return fmaxf(fmaxf(x, y), z); }

// max that keeps NaN
__device__ __forceinline__ float max3nan(float x, float y, float z) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

#ifndef KVQ_RD
#define KVQ_RD 88
#define KVQ_RI 208
#endif
#ifndef KVQ_KT
#define KVQ_KT 128
#endif
// Shapes per head size.  kQT query tiles of 128 rows share the key tiles that
// the CTA loads, one softmax warpgroup each; TMEM holds two score tiles and
// one output tile per query tile.
template <int D>
struct Geom {
  static constexpr int kQT = D == 256 ? 1 : 2;
  static constexpr int kKeys = D == 256 ? 64 : KVQ_KT;   // keys per tile
  static constexpr int kNB = kKeys == 64 ? 2 : 1;        // score tiles per query tile in TMEM
  static constexpr int kSlot = kKeys * D * 2;            // one K or V tile
  static constexpr int kSlots = D == 256 ? 5 : (D == 128 ? 8 * 64 / kKeys : 8);
  static constexpr int kSoftmax = kQT * 128;             // softmax threads
  static constexpr int kThreads = kSoftmax + 128;        // + MMA, load, V guard and unit warps
  static constexpr int kQTile = kRows * D * 2;
  static constexpr int kQ = 0;
  static constexpr int kKV = kQ + kQT * kQTile;
  static constexpr int kStat = kKV + kSlots * kSlot;     // float m[128], w[128] per query tile (masses)
  static constexpr int kBar = kStat + kQT * 2 * kRows * 4;
  static constexpr int kMisc = kBar + 400;
  static constexpr int kSmem = kMisc + 128 + 1024;       // + alignment slack
  static_assert(kSmem <= 232448, "shared memory per block");
  // TMEM columns
  static constexpr int kS = 0, kO = kNB * kQT * kKeys;
  static_assert(kO + kQT * D <= 512, "TMEM columns");
};

// mbarriers, 8 bytes each, from Geom::kBar on
enum : int {
  kBarQFull = 0,         // the unit's Q tiles have landed
  kBarQEmpty,            // its last score MMA has read them
  kBarS,                 // [2 x query tile + buffer] a score tile is in TMEM
  kBarP = kBarS + 4,     // [same] its P is in TMEM (one arrival per softmax warp)
  kBarH = kBarP + 4,     // [same] the first half of its P is
  kBarO = kBarH + 4,     // [query tile + buffer] a PV MMA is done
  kBarG = kBarO + 2,     // V of an edge tile has landed: the guard may look at it
  kBarV,                 // the guard is done with it
  kBarUFull,             // [2] a unit is published
  kBarUEmpty = kBarUFull + 2,  // [2] every warp is done with it
  kBarDrain = kBarUEmpty + 2,
  kBarKVFull,            // [kSlots], then [kSlots] empty
  kBarCount = kBarKVFull + 24
};
static_assert(kBarCount * 8 <= 400, "barriers fit");

struct Shared {  // at Geom::kMisc
  uint32_t tmem;
  int stop;
  int odd_v[2];   // per unit slot: V values of an edge tile were left out
  Unit unit[2];
};

// A running position in a ring of barriers
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// The key tiles of a unit's query tile q: tokens [i0 + q W1, ...) of n
template <int KT>
__device__ __forceinline__ int key_tiles(int i0, int q, int W1, int n) {
  const int first = i0 + q * W1;
  return first < n ? (min(n, first + W1) + KT - 1) / KT : 0;
}

template <int D, bool MASS>
__global__ void __launch_bounds__(Geom<D>::kThreads, 1) prompt_kernel(const __grid_constant__ CUtensorMap mq,
                                                                      const __grid_constant__ CUtensorMap mk,
                                                                      const __grid_constant__ CUtensorMap mv,
                                                                      const __grid_constant__ PromptDev pd) {
  using Geo = Geom<D>;
  constexpr int QT = Geo::kQT, NS = Geo::kSlots, KT = Geo::kKeys, NB = Geo::kNB;
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

  // rows of the Q tiles that no box fills (g not a divisor of 128) stay zero
  for (int i = tid; i < QT * Geo::kQTile / 16; i += Geo::kThreads)
    reinterpret_cast<uint4*>(smem + Geo::kQ)[i] = make_uint4(0, 0, 0, 0);
  fence_async_smem();
  if (tid == 0) {
    mbar_init(bar(kBarQFull), 1);
    mbar_init(bar(kBarQEmpty), 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(kBarS + i), 1);
      mbar_init(bar(kBarP + i), 4);
      mbar_init(bar(kBarH + i), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarO + i), 1);
      mbar_init(bar(kBarUFull + i), 1);
      mbar_init(bar(kBarUEmpty + i), 4 * QT + 3);
    }
    mbar_init(bar(kBarG), 1);
    mbar_init(bar(kBarV), 1);
    mbar_init(bar(kBarDrain), 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(bar(kBarKVFull + i), 1);
      mbar_init(bar(kBarKVFull + NS + i), 1);
    }
    mbar_init_fence();
    sh->stop = 0;
  }
  if (warp == 0) tmem_alloc512(smem_u32(&sh->tmem));
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = sh->tmem;

  if (warp >= 4 * QT) {
    if constexpr (QT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(KVQ_RD));
    const int role = warp - 4 * QT;
    if (role == 3) {
      // ------------------------------------------------------------ units
      if (blockIdx.x == 0) {
        for (int s = lane; s < a.num_seqs; s += 32) {
          const int f = a.cu_seqlens[s], e = a.cu_seqlens[s + 1];
          if (f < 0 || e < f || e > a.total_tokens || e - f > a.max_seq_tokens)
            report_error(a.dev_status, KVQ_ERR_DEVICE_BOUNDS);
        }
      }
      Ring r;
      for (int round = 0;; ++round) {
        const long long ul = static_cast<long long>(round) * gridDim.x +
                             ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        Unit u{0, 0, 0, -1, 0};  // n = -1: no more
        if (ul < pd.units) {
          u = locate_unit(pd, static_cast<int>(ul), lane);
          if (u.n == 0) {
            if (a.num_seqs > kSortedSeqs) continue;
            u.n = -1;
          }
        }
        if (!warp_wait(bar(kBarUEmpty + r.slot), r.phase ^ 1u, stop)) break;
        if (lane == 0) {
          sh->unit[r.slot] = u;
          sh->odd_v[r.slot] = 0;
          mbar_arrive(bar(kBarUFull + r.slot));
        }
        r.next(2);
        if (u.n < 0) break;
      }
    } else if (role == 1) {
      // ------------------------------------------------------------ loads
      if (lane == 0) {
        Ring ru, kv;
        uint32_t ph_q = 0;
        bool ok = true;
        int issued = 0;
        while (ok) {
          if (!mbar_wait(bar(kBarUFull + ru.slot), ru.phase, stop)) break;
          const Unit u = sh->unit[ru.slot];
          mbar_arrive(bar(kBarUEmpty + ru.slot));
          ru.next(2);
          if (u.n < 0) break;
          const int i0 = u.run * W1 * QT;
          int nk = 0;
          for (int q = 0; q < QT; ++q) nk = max(nk, key_tiles<KT>(i0, q, W1, u.n));
          if (!(ok = mbar_wait(bar(kBarQEmpty), ph_q ^ 1u, stop))) break;
          ph_q ^= 1u;
          mbar_expect_tx(bar(kBarQFull), QT * W1 * G * D * 2);
          for (int q = 0; q < QT; ++q)
            for (int c = 0; c < D / 64; ++c)
              tma_load(s0 + Geo::kQ + q * Geo::kQTile + c * kRows * 128, &mq, 64 * c, u.head * G,
                       u.first + i0 + q * W1, bar(kBarQFull));
          // in the order the MMA warp takes them: K0 .. K(NB-1) V0 K(NB) V1 ...
          auto load = [&](const CUtensorMap* map, int j) {
            if (!ok || j >= nk || !(ok = mbar_wait(bar(kBarKVFull + NS + kv.slot), kv.phase ^ 1u, stop))) return;
            mbar_expect_tx(bar(kBarKVFull + kv.slot), Geo::kSlot);
            for (int c = 0; c < D / 64; ++c)
              tma_load(s0 + Geo::kKV + kv.slot * Geo::kSlot + c * KT * 128, map, 64 * c, u.head, u.first + j * KT,
                       bar(kBarKVFull + kv.slot));
            kv.next(NS);
            issued = min(issued + 1, NS);
          };
          for (int j = 0; j < NB; ++j) load(&mk, j);
          for (int j = 0; j < nk && ok; ++j) {
            load(&mv, j);
            load(&mk, j + NB);
          }
        }
        if (*stop) {  // copies in flight land before the shared memory is given back
          const long long t0 = global_ns();
          for (int i = 0; i < issued; ++i) {
            kv.slot = kv.slot == 0 ? NS - 1 : kv.slot - 1;
            if (kv.slot == NS - 1) kv.phase ^= 1u;
            while (!mbar_try(bar(kBarKVFull + kv.slot), kv.phase) && global_ns() - t0 < kWaitLimitNs) {
            }
          }
          while (issued > 0 && !mbar_try(bar(kBarQFull), ph_q ^ 1u) && global_ns() - t0 < kWaitLimitNs) {
          }
        }
      }
    } else if (role == 0) {
      // ------------------------------------------------------------ matrix instructions
      // The whole warp runs this, on values it knows to be uniform, and one
      // elected lane issues: descriptors then stay in uniform registers (from
      // a single-lane branch each instruction took about 70 cycles to issue).
      Ring ru, kv;
      uint32_t ph_q = 0, ph_p = 0, ph_v = 0;  // ph_p: a bit per P buffer
      bool ok = true;
      const bool leader = elect_one();
      const uint64_t dq = sw128_desc(s0 + Geo::kQ, 0), dk = sw128_desc(s0 + Geo::kKV, 0);
      const uint64_t dv = sw128_desc(s0 + Geo::kKV, KT * 128);
      auto commit = [&](int b) {
        if (leader) mma_commit(bar(b));
      };
      // score tile j of query tile q: S = Q_q K^T with K in slot `slot`
      auto score = [&](int q, int j, int slot) {
        const int b = 2 * q + j % NB;
        const uint64_t qa = dq + (q * Geo::kQTile >> 4), ka = dk + (slot * Geo::kSlot >> 4);
        if (leader) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(tm + Geo::kS + (NB * q + j % NB) * KT, qa + (((k >> 2) * kRows * 128 + (k & 3) * 32) >> 4),
                   ka + (((k >> 2) * KT * 128 + (k & 3) * 32) >> 4), idesc_m128(KT, false), k != 0);
          mma_commit(bar(kBarS + b));
        }
      };
      // O_q (+)= P V with V in slot `slot`, half h of the keys
      auto value = [&](int q, int j, int slot, int h) {
        const uint64_t va = dv + (slot * Geo::kSlot >> 4);
        if (leader) {
#pragma unroll
          for (int k = h * KT / 32; k < (h + 1) * KT / 32; ++k)
            mma_ts(tm + Geo::kO + q * D, tm + Geo::kS + (NB * q + j % NB) * KT + 8 * k, va + (k * 2048 >> 4), idesc_m128(D, true),
                   j > 0 || k > 0);
          if (h == 1) mma_commit(bar(kBarO + q + j % NB));
        }
      };
      auto wait_kv = [&] {
        const bool r = warp_wait(bar(kBarKVFull + kv.slot), kv.phase, stop);
        fence_after();
        return r;
      };
      while (ok) {
        if (!warp_wait(bar(kBarUFull + ru.slot), ru.phase, stop)) break;
        const int n = __shfl_sync(kFull, sh->unit[ru.slot].n, 0);
        const int i0 = __shfl_sync(kFull, sh->unit[ru.slot].run, 0) * W1 * QT, edge = i0 / KT;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarUEmpty + ru.slot));
        ru.next(2);
        if (n < 0) break;
        const int nkq[2] = {key_tiles<KT>(i0, 0, W1, n), QT == 2 ? key_tiles<KT>(i0, 1, W1, n) : 0};
        const int nk = max(nkq[0], nkq[1]);
        if (!(ok = warp_wait(bar(kBarQFull), ph_q, stop))) break;
        ph_q ^= 1u;
        // the first NB score tiles; later ones follow the PV that frees their buffer
        for (int j = 0; j < min(nk, NB); ++j) {
          if (!(ok = wait_kv())) break;
#pragma unroll
          for (int q = 0; q < QT; ++q)
            if (j < nkq[q]) score(q, j, kv.slot);
          commit(kBarKVFull + NS + kv.slot);
          kv.next(NS);
        }
        if (!ok) break;
        if (nk <= NB) commit(kBarQEmpty);
        for (int j = 0; j < nk; ++j) {
          const int vslot = kv.slot;
          if (!(ok = wait_kv())) break;
          kv.next(NS);
          bool guarded = j >= edge;  // the guard looks at V while the softmax of the tile runs
          if (guarded && lane == 0) mbar_arrive(bar(kBarG));
          bool have_k = false;
#pragma unroll
          for (int q = 0; q < QT; ++q) {
            if (!ok || j >= nkq[q]) continue;
            const int b = 2 * q + j % NB;
            ok = warp_wait(bar(kBarH + b), (ph_p >> b) & 1u, stop);
            if (ok && guarded) {
              ok = warp_wait(bar(kBarV), ph_v, stop);
              ph_v ^= 1u;
              guarded = false;
            }
            fence_after();
            if (!ok) continue;
            value(q, j, vslot, 0);
            if (!(ok = warp_wait(bar(kBarP + b), (ph_p >> b) & 1u, stop))) continue;
            ph_p ^= 1u << b;
            fence_after();
            value(q, j, vslot, 1);
            if (j + NB < nkq[q]) {
              if (!have_k && !(ok = wait_kv())) continue;
              have_k = true;
              score(q, j + NB, kv.slot);
            }
          }
          if (!ok) break;
          commit(kBarKVFull + NS + vslot);
          if (j + NB < nk) {
            commit(kBarKVFull + NS + kv.slot);
            if (j + NB + 1 == nk) commit(kBarQEmpty);
            kv.next(NS);
          }
        }
      }
      if (*stop && leader) {  // matrix instructions in flight end before TMEM is freed
        mma_commit(bar(kBarDrain));
        const long long t0 = global_ns();
        while (!mbar_try(bar(kBarDrain), 0) && global_ns() - t0 < kWaitLimitNs) {
        }
      }
    } else {
      // ------------------------------------------------------------ V guard
      // V of the tiles that hold keys some row does not see: rows past the
      // sequence and values that are not finite become zero
      Ring ru, kv;
      uint32_t ph_g = 0;
      while (warp_wait(bar(kBarUFull + ru.slot), ru.phase, stop)) {
        const Unit u = sh->unit[ru.slot];
        const int uslot = ru.slot;
        ru.next(2);
        if (u.n < 0) break;
        const int i0 = u.run * W1 * QT, edge = i0 / KT;
        int nk = 0;
        for (int q = 0; q < QT; ++q) nk = max(nk, key_tiles<KT>(i0, q, W1, u.n));
        bool ok = true;
        for (int j = 0; j < min(nk, NB); ++j) kv.next(NS);  // K
        for (int j = 0; j < nk; ++j) {
          if (j >= edge) {
            if (!(ok = warp_wait(bar(kBarG), ph_g, stop))) break;
            ph_g ^= 1u;
            uint4* p = reinterpret_cast<uint4*>(smem + Geo::kKV + kv.slot * Geo::kSlot);
            bool odd = false;
#pragma unroll 4
            for (int i = lane; i < Geo::kSlot / 16; i += 32) {
              const int key = j * KT + ((i >> 3) % KT);
              uint4 x = p[i];
              if (key >= u.n) {
                p[i] = make_uint4(0, 0, 0, 0);
                continue;
              }
              uint32_t* w = reinterpret_cast<uint32_t*>(&x);
              bool bad = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((w[e] & 0x7C00u) == 0x7C00u) { w[e] &= 0xFFFF0000u; bad = true; }
                if ((w[e] & 0x7C000000u) == 0x7C000000u) { w[e] &= 0x0000FFFFu; bad = true; }
              }
              if (bad) {
                p[i] = x;
                odd = true;
              }
            }
            if (odd) sh->odd_v[uslot] = 1;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarV));
          }
          kv.next(NS);                   // V
          if (j + NB < nk) kv.next(NS);  // K
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(bar(kBarUEmpty + uslot));
      }
    }
  } else {
    // -------------------------------------------------------------- softmax
    if constexpr (QT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(KVQ_RI));
    const int q = warp >> 2, row = tid & 127;
    const uint32_t tlane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tO = tm + Geo::kO + q * D + tlane;
    const int T = a.cfg.tile_tokens, wid = min(T, KT), ent = KT / wid;  // keys per mass entry, entries per tile
    float* s_m = reinterpret_cast<float*>(smem + Geo::kStat) + q * 2 * kRows;
    float* s_w = s_m + kRows;
    Ring ru;
    uint32_t ph_s[2] = {0u, 0u}, ph_o[2] = {0u, 0u};
    const bool leader = elect_one();
    constexpr int HK = KT / 2;  // keys of half a tile
    while (true) {
      if (!warp_wait(bar(kBarUFull + ru.slot), ru.phase, stop)) break;
      const Unit u = sh->unit[ru.slot];
      const int uslot = ru.slot;
      ru.next(2);
      if (u.n < 0) break;
      const int first = u.run * W1 * QT + q * W1;        // the tile's first token
      const int nk = key_tiles<KT>(first, 0, W1, u.n);
      const int ti = first + row / G;                    // this row's token
      const bool live = row < W1 * G && ti < u.n;
      const int vis = live ? ti : u.n - 1;               // last key this row sees
      const int masked = first / KT;                     // tiles from here on need the mask
      const long long slot = MASS && nk > 0 ? mass_slot(pd, u, u.run * QT + q) : -1;
      float* scr = pd.scratch + (static_cast<size_t>(blockIdx.x) * QT + q) * pd.max_tiles_k * (ent + 1) * kRows + row;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < nk; ++j) {
        const int buf = j % NB;
        const uint32_t tS = tm + Geo::kS + (NB * q + buf) * KT + tlane;
        if (!(ok = warp_wait(bar(kBarS + 2 * q + buf), ph_s[buf], stop))) break;
        ph_s[buf] ^= 1u;
        fence_after();
        // The tile goes in two halves.  The first half's weights are taken
        // relative to the maximum up to it while the second half's scores are
        // still on their way and being compared; P V starts on them while the
        // second half's weights are computed.
        float s[KT];
        const int lim = vis - j * KT;  // last key of the tile that the row sees
        // loads of half h, its mask and maximum (times the scale)
        auto load = [&](auto at) {
          constexpr int o = decltype(at)::value;
          tmem_ld32<o>(tS + o, s);
          if constexpr (HK == 64) tmem_ld32<o + HK - 32>(tS + o + 32, s);
        };
        auto top_of = [&](auto at) {
          constexpr int o = decltype(at)::value;
          tmem_wait32<o>(s);
          if constexpr (HK == 64) tmem_wait32<o + HK - 32>(s);
          if (j >= masked) {
#pragma unroll
            for (int c = o; c < o + HK; ++c) s[c] = c <= lim ? s[c] : -INFINITY;
          }
          float mx[4] = {s[o], s[o + 1], s[o + 2], s[o + 3]};
#pragma unroll
          for (int c = o + 4; c < o + HK - 4; c += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = max3nan(mx[e], s[c + e], s[c + 4 + e]);
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3nan(mx[e], s[o + HK - 4 + e], s[o + HK - 4 + e]);
          const float t = max3nan(mx[0], mx[1], max3nan(mx[2], mx[3], mx[3])) * pd.qscale;
          if (!(t < INFINITY)) l = NAN;  // a NaN or an infinite score: the row is NaN
          return t;
        };
        // The maximum moves to `top` in the lanes where it is more than kLazy
        // larger (m = -inf before the first finite score); O and l follow.
        auto grow = [&](float top) {
          float alpha = 1.f;
          if (top > m + kLazy) {
            alpha = ex2(m - top);
            m = top;
            l *= alpha;
          }
          if (j == 0) return true;
          // the last PV is done: with one score buffer this tile's score MMA came after it
          if (NB > 1 && !warp_wait(bar(kBarO + q + (j - 1) % NB), ph_o[(j - 1) % NB] ^ 1u, stop)) return false;
          fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 8) {  // few registers: the scores stay in theirs
            float o[8];
            tmem_ld8(tO + c, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= alpha;
            tmem_st8(tO + c, o);
          }
          return true;
        };
        float2 part[KT / 32];  // sums of 32 keys
        uint32_t p[HK / 2];
        auto weigh = [&](auto at) {
          constexpr int o = decltype(at)::value;
          const float mu = m == -INFINITY ? 0.f : m;  // a row with no finite score so far
          const float2 sc2 = make_float2(pd.qscale, pd.qscale), mu2 = make_float2(-mu, -mu);
#pragma unroll
          for (int c = 0; c < HK; c += 2) {
            const float2 x = __ffma2_rn(make_float2(s[o + c], s[o + c + 1]), sc2, mu2);
            const float2 e = make_float2(ex2(x.x), ex2(x.y));
            float2& sum = part[(o + c) / 32];
            sum = c % 32 == 0 ? e : __fadd2_rn(sum, e);
            p[c / 2] = h2_as_u32(__float22half2_rn(e));
          }
        };
        // P of 32 keys takes 16 columns of scores already read
        auto store = [&](int o) {
          if constexpr (HK == 64) tmem_st32<0>(tS + o / 2, p); else tmem_st16(tS + o / 2, p);
          tmem_wait_st();
          fence_before();
          __syncwarp();
        };
        constexpr std::integral_constant<int, 0> kFirst{};
        constexpr std::integral_constant<int, HK> kSecond{};
        load(kFirst);
        float top = top_of(kFirst);
        load(kSecond);
        if (__any_sync(kFull, top > m + kLazy) && !(ok = grow(top))) break;
        weigh(kFirst);
        top = top_of(kSecond);
        if (__any_sync(kFull, top > m + kLazy)) {  // rare: the first half again
          if (!(ok = grow(top))) break;
          weigh(kFirst);
        }
        store(0);
        mbar_arrive_if(leader, bar(kBarH + 2 * q + buf));
        weigh(kSecond);
        store(HK);
        mbar_arrive_if(leader, bar(kBarP + 2 * q + buf));
        ph_o[j % NB] ^= 1u;
        const float mu = m == -INFINITY ? 0.f : m;
        float ps[KT / 32];
        float all = 0.f;
#pragma unroll
        for (int k = 0; k < KT / 32; ++k) all += ps[k] = part[k].x + part[k].y;
        l += all;
        if (MASS && slot >= 0) {
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
      if (!ok) break;
      if (nk > 0) {
        // ---- the tile's rows
        if (!warp_wait(bar(kBarO + q + (nk - 1) % NB), ph_o[(nk - 1) % NB] ^ 1u, stop)) break;
        fence_after();
        const bool odd = *static_cast<volatile int*>(&sh->odd_v[uslot]) != 0;
        const float inv = 1.f / l;
        const size_t orow = static_cast<size_t>(u.first + (live ? ti : 0)) * nh * G + u.head * G + row % G;
        __half* out = static_cast<__half*>(a.out) + orow * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32<0>(tO + c, o);
          tmem_wait32<0>(o);
          if (!live) continue;
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= inv;
          if (odd) {  // the values the V guard left out, to the rows that see them
            for (int key = u.run * W1 * QT / KT * KT; key <= vis; ++key) {
              const __half* vr = static_cast<const __half*>(a.v) + static_cast<size_t>(u.first + key) * a.v_stride +
                                 u.head * D + c;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float x = __half2float(vr[e]);
                if (!(fabsf(x) <= 65504.f)) o[e] += x;
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 w;
            w.x = h2_as_u32(__floats2half2_rn(o[e], o[e + 1]));
            w.y = h2_as_u32(__floats2half2_rn(o[e + 2], o[e + 3]));
            w.z = h2_as_u32(__floats2half2_rn(o[e + 4], o[e + 5]));
            w.w = h2_as_u32(__floats2half2_rn(o[e + 6], o[e + 7]));
            *reinterpret_cast<uint4*>(out + c + e) = w;
          }
        }
        if (live && a.lse != nullptr) a.lse[orow] = (m + log2f(l)) * 0.6931471805599453f;
        if (MASS && slot >= 0) {
          const bool counts = live && (a.mass_window == 0 || ti >= u.n - a.mass_window);
          s_m[row] = m == -INFINITY ? 0.f : m;
          s_w[row] = counts ? inv : 0.f;
          asm volatile("bar.sync %0, 128;" ::"r"(1 + q) : "memory");
          float* dst = pd.part + static_cast<size_t>(slot) * pd.max_tiles_k * ent;
          const float* base = scr - row;
          for (int i = row; i < nk * ent; i += kRows) {
            const float* psum = base + (static_cast<size_t>(i / ent) * (ent + 1) + i % ent) * kRows;
            const float* pm = base + (static_cast<size_t>(i / ent) * (ent + 1) + ent) * kRows;
            float sum = 0.f;
#pragma unroll 4
            for (int r = 0; r < kRows; r += 4) {
              const float4 x = *reinterpret_cast<const float4*>(psum + r), y = *reinterpret_cast<const float4*>(pm + r);
              const float4 f = *reinterpret_cast<const float4*>(s_m + r), w = *reinterpret_cast<const float4*>(s_w + r);
              if (w.x != 0.f) sum += x.x * ex2(y.x - f.x) * w.x;
              if (w.y != 0.f) sum += x.y * ex2(y.y - f.y) * w.y;
              if (w.z != 0.f) sum += x.z * ex2(y.z - f.z) * w.z;
              if (w.w != 0.f) sum += x.w * ex2(y.w - f.w) * w.w;
            }
            dst[i] = sum;
          }
          asm volatile("bar.sync %0, 128;" ::"r"(1 + q) : "memory");
        }
        fence_before();
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
// tile t.  A CTA per 32 tiles: lanes over the tiles, warps over the (run,
// head) rows with a fixed stride, then the warps in order.
constexpr int kMassWarps = 32;
__global__ void __launch_bounds__(kMassWarps * 32) prompt_mass_kernel(PromptDev pd, int KT) {
  __shared__ float s_sum[kMassWarps][33];
  const PromptArgs& a = pd.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = blockIdx.y, t = blockIdx.x * 32 + lane;
  const int T = a.cfg.tile_tokens, W1 = pd.tile_tokens, nh = a.cfg.num_kv_heads;
  const int wid = min(T, KT), per = T / wid;  // partial sums per tile of T
  Unit u{s, 0, 0, 0, 0};
  u.n = seq_len(a, s, u.first);
  const int tiles = min((u.n + T - 1) / T, a.max_tiles);
  if (blockIdx.x * 32 >= tiles) return;
  const int w0 = a.mass_window == 0 ? 0 : max(0, u.n - a.mass_window) / W1;
  const int r0 = max(w0, blockIdx.x * 32 * T / W1), rows = (u.n + W1 - 1) / W1 * nh;
  const size_t stride = static_cast<size_t>(pd.max_tiles_k) * (KT / wid);
  float sum = 0.f;
#pragma unroll 4
  for (int x = r0 * nh + warp; x < rows; x += kMassWarps) {
    u.head = x % nh;
    const int run = x / nh;
    // the key tiles this query tile went over
    const int held = (min(u.n, (run + 1) * W1) + KT - 1) / KT * (KT / wid);
    const float* p = pd.part + static_cast<size_t>(mass_slot(pd, u, run)) * stride;
    for (int k = 0; k < per; ++k)
      if (t < tiles && t * per + k < held) sum += p[t * per + k];
  }
  s_sum[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && t < tiles) {
    sum = 0.f;
    for (int w = 0; w < kMassWarps; ++w) sum += s_sum[w][lane];
    a.mass[static_cast<size_t>(s) * a.max_tiles + t] += sum;
  }
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
int key_tile(const kvq_config& cfg) { return cfg.head_dim == 256 ? Geom<256>::kKeys : Geom<128>::kKeys; }
static_assert(Geom<64>::kKeys == Geom<128>::kKeys, "key tiles of d = 64");
int query_tiles(const kvq_config& cfg) { return cfg.head_dim == 256 ? Geom<256>::kQT : Geom<128>::kQT; }
struct PromptSizes {
  long long units;
  int max_tiles_k, window_runs, grid;
  size_t scratch_floats, part_floats;
};
PromptSizes prompt_sizes(const kvq_config& cfg, int num_seqs, int total_tokens, int max_seq_tokens, int window,
                         int sms) {
  PromptSizes z;
  const int W1 = tile_tokens(cfg), keys = key_tile(cfg), ent = keys / std::min(keys, cfg.tile_tokens);
  z.units = prompt_units(cfg, num_seqs, total_tokens);
  z.max_tiles_k = (max_seq_tokens + keys - 1) / keys;
  z.window_runs = window == 0 ? 0 : std::min((window - 1) / W1 + 2, (max_seq_tokens + W1 - 1) / W1);
  z.grid = static_cast<int>(std::min<long long>(z.units, sms));
  z.scratch_floats = static_cast<size_t>(z.grid) * query_tiles(cfg) * z.max_tiles_k * (ent + 1) * kRows;
  const size_t runs = window == 0 ? static_cast<size_t>(total_tokens) / W1 + num_seqs
                                  : static_cast<size_t>(num_seqs) * z.window_runs;
  z.part_floats = runs * cfg.num_kv_heads * z.max_tiles_k * ent;
  return z;
}

template <int D, bool MASS>
cudaError_t launch_prompt(const PromptArgs& a, cudaStream_t s) {
  using Geo = Geom<D>;
  static PerDevice known;  // the shared memory is opted in to once per device
  auto kern = prompt_kernel<D, MASS>;
  int sms = 0;
  cudaError_t e = known.get(&sms, [&](int* v) {
    const cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo::kSmem);
    return r != cudaSuccess ? r : device_sm_count(v);
  });
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
  pd.unit_tokens = pd.tile_tokens * Geo::kQT;
  pd.units = static_cast<int>(z.units);
  pd.max_tiles_k = z.max_tiles_k;
  pd.window_runs = z.window_runs;
  pd.qscale = a.softmax_scale * kLog2e;
  pd.scratch = static_cast<float*>(a.workspace);
  pd.part = pd.scratch + z.scratch_floats;
  kern<<<z.grid, Geo::kThreads, Geo::kSmem, s>>>(mq, mk, mv, pd);
  e = cudaGetLastError();
  if (e != cudaSuccess || !MASS) return e;
  const int tiles = std::min(a.max_tiles, (a.max_seq_tokens + a.cfg.tile_tokens - 1) / a.cfg.tile_tokens);
  prompt_mass_kernel<<<dim3((tiles + 31) / 32, a.num_seqs), kMassWarps * 32, 0, s>>>(pd, Geo::kKeys);
  return cudaGetLastError();
}

}  // namespace

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
