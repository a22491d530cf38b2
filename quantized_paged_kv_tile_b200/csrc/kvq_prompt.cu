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

#include "kvq_device.cuh"
#include "kvq_sm100.cuh"

namespace kvq {

namespace {

using namespace sm100;

constexpr int kRows = 128;    // query rows per unit (TMEM lanes)
constexpr int kKeys = 128;    // keys per tile
constexpr int kThreads = 128;
// up to this many sequences the units are taken longest first
constexpr int kSortedSeqs = 1024;

struct PromptDev {
  PromptArgs a;
  int unit_tokens;     // query tokens per unit
  int units;           // host bound on the number of units
  int max_tiles_k;     // key tiles of the longest sequence
  int window_units;    // units per (sequence, head) that can hold counted queries; 0: all
  float qscale;        // softmax_scale * log2 e
  float* scratch;      // per CTA [max_tiles_k][kKeys / T + 1][kRows]
  float* part;         // per unit [max_tiles_k * kKeys / T]
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

// slot of a unit in the partial masses; -1: none of its queries counts
__device__ __forceinline__ long long mass_slot(const PromptDev& pd, const Unit& u) {
  const PromptArgs& a = pd.a;
  const int W = pd.unit_tokens;
  if (a.mass_window == 0)
    return (static_cast<long long>(u.first / W + u.seq + u.run)) * a.cfg.num_kv_heads + u.head;
  const int r0 = max(0, u.n - a.mass_window) / W;
  if (u.run < r0) return -1;
  return (static_cast<long long>(u.seq) * pd.window_units + (u.run - r0)) * a.cfg.num_kv_heads + u.head;
}

template <int D>
struct Geom {
  static constexpr int kQ = 0;                          // Q: 128 rows x D, 64-channel blocks of 16 KB
  static constexpr int kK = kQ + kRows * D * 2;         // K tile: 128 keys x D
  static constexpr int kV = kK + kKeys * D * 2;         // V tile: 128 keys x D
  static constexpr int kStat = kV + kKeys * D * 2;      // float m[128], w[128]
  static constexpr int kBar = kStat + 2 * kRows * 4;    // mbarriers: q, kv, mma
  static constexpr int kMisc = kBar + 32;               // TMEM slot, stop flag, non-finite V flag, unit
  static constexpr int kSmem = kMisc + 64 + 1024;       // + alignment slack
};

template <int D, bool MASS>
__global__ void __launch_bounds__(kThreads) prompt_kernel(const __grid_constant__ CUtensorMap mq,
                                                          const __grid_constant__ CUtensorMap mk,
                                                          const __grid_constant__ CUtensorMap mv, PromptDev pd) {
  using Geo = Geom<D>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const PromptArgs& a = pd.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = a.cfg.group_size, nh = a.cfg.num_kv_heads, T = a.cfg.tile_tokens;
  const int W = pd.unit_tokens, row = tid;
  const uint32_t s0 = smem_u32(smem), bar_q = s0 + Geo::kBar, bar_kv = bar_q + 8, bar_mma = bar_q + 16;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + Geo::kMisc);
  volatile int* stop = reinterpret_cast<volatile int*>(smem + Geo::kMisc + 4);
  int* odd_v = reinterpret_cast<int*>(smem + Geo::kMisc + 8);
  Unit* s_unit = reinterpret_cast<Unit*>(smem + Geo::kMisc + 16);
  float* s_m = reinterpret_cast<float*>(smem + Geo::kStat);
  float* s_w = s_m + kRows;

  // rows of the Q tile that no box fills (g not a divisor of 128) stay zero
  for (int i = tid; i < kRows * D * 2 / 16; i += kThreads)
    reinterpret_cast<uint4*>(smem + Geo::kQ)[i] = make_uint4(0, 0, 0, 0);
  fence_async_smem();
  if (tid == 0) {
    mbar_init(bar_q, 1);
    mbar_init(bar_kv, 1);
    mbar_init(bar_mma, 1);
    mbar_init_fence();
    *stop = 0;
    *odd_v = 0;
  }
  if (warp == 0) tmem_alloc512(smem_u32(tslot));
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = *tslot, tS = tm, tO = tm + kKeys;  // S (and P over it): 128 columns; O: D columns
  const uint32_t tlane = static_cast<uint32_t>(warp * 32) << 16;

  if (blockIdx.x == 0) {
    for (int s = tid; s < a.num_seqs; s += kThreads) {
      const int f = a.cu_seqlens[s], e = a.cu_seqlens[s + 1];
      if (f < 0 || e < f || e > a.total_tokens || e - f > a.max_seq_tokens)
        report_error(a.dev_status, KVQ_ERR_DEVICE_BOUNDS);
    }
  }

  uint32_t ph_q = 0, ph_kv = 0, ph_mma = 0;
  bool failed = false;
  const int sub_n = kKeys / T;
  for (int round = 0; !failed; ++round) {
    const long long ul = static_cast<long long>(round) * gridDim.x +
                         ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    if (ul >= pd.units) break;
    if (warp == 0) {
      const Unit u = locate_unit(pd, static_cast<int>(ul), lane);
      if (lane == 0) *s_unit = u;
    }
    __syncthreads();
    const Unit u = *s_unit;
    __syncthreads();
    if (u.n == 0) {
      if (a.num_seqs <= kSortedSeqs) break;
      continue;
    }
    const int i0 = u.run * W, i1 = min(u.n, i0 + W);  // query tokens [i0, i1)
    const int nk = (i1 + kKeys - 1) / kKeys;          // key tiles
    const int edge = i0 / kKeys;                      // tiles from here on hold keys that some row does not see
    const int ti = i0 + row / G;                      // this row's token
    const bool live = row < W * G && ti < u.n;
    const int vis = live ? ti : i1 - 1;               // last key this row sees
    const long long slot = MASS ? mass_slot(pd, u) : -1;
    float* scr = pd.scratch + static_cast<size_t>(blockIdx.x) * pd.max_tiles_k * (sub_n + 1) * kRows;
    float m = -INFINITY, l = 0.f;
    if (tid == 0) {
      mbar_expect_tx(bar_q, W * G * D * 2);
      for (int c = 0; c < D / 64; ++c)
        tma_load(s0 + Geo::kQ + c * kRows * 128, &mq, 64 * c, u.head * G, u.first + i0, bar_q);
    }
    for (int j = 0; j < nk; ++j) {
      if (tid == 0) {
        mbar_expect_tx(bar_kv, 2 * kKeys * D * 2);
        for (int c = 0; c < D / 64; ++c) {
          tma_load(s0 + Geo::kK + c * kKeys * 128, &mk, 64 * c, u.head, u.first + j * kKeys, bar_kv);
          tma_load(s0 + Geo::kV + c * kKeys * 128, &mv, 64 * c, u.head, u.first + j * kKeys, bar_kv);
        }
      }
      bool ok = j > 0 || mbar_wait(bar_q, ph_q, stop);
      ok = ok && mbar_wait(bar_kv, ph_kv, stop);
      if (__syncthreads_or(!ok)) {
        failed = true;
        break;
      }
      ph_kv ^= 1;
      if (tid == 0) {
        fence_after();
        for (int k = 0; k < D / 16; ++k)
          mma_ss(tS, sw128_desc(s0 + Geo::kQ + (k >> 2) * kRows * 128 + (k & 3) * 32, 0),
                 sw128_desc(s0 + Geo::kK + (k >> 2) * kKeys * 128 + (k & 3) * 32, 0), idesc_m128(kKeys, false), k != 0);
        mma_commit(bar_mma);
      }
      if (j >= edge) {
        // V of a tile with masked keys: rows past the sequence and values that
        // are not finite become zero (the latter are added at the end)
        for (int i = tid; i < kKeys * D / 8; i += kThreads) {
          const int key = (i >> 3) % kKeys;
          uint4* p = reinterpret_cast<uint4*>(smem + Geo::kV) + i;
          uint4 x = *p;
          if (j * kKeys + key >= u.n) {
            *p = make_uint4(0, 0, 0, 0);
          } else {
            uint32_t* w = reinterpret_cast<uint32_t*>(&x);
            bool odd = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((w[e] & 0x7C00u) == 0x7C00u) { w[e] &= 0xFFFF0000u; odd = true; }
              if ((w[e] & 0x7C000000u) == 0x7C000000u) { w[e] &= 0x0000FFFFu; odd = true; }
            }
            if (odd) {
              *p = x;
              *odd_v = 1;
            }
          }
        }
        fence_async_smem();
      }
      ok = mbar_wait(bar_mma, ph_mma, stop);
      if (__syncthreads_or(!ok)) {
        failed = true;
        break;
      }
      ph_mma ^= 1;
      fence_after();

      float s[kKeys];
      tmem_ld32<0>(tS + tlane, s);
      tmem_ld32<32>(tS + tlane + 32, s);
      tmem_ld32<64>(tS + tlane + 64, s);
      tmem_ld32<96>(tS + tlane + 96, s);
      tmem_wait32<0>(s);
      tmem_wait32<32>(s);
      tmem_wait32<64>(s);
      tmem_wait32<96>(s);
      if (j >= edge) {
        const int lim = vis - j * kKeys;
#pragma unroll
        for (int c = 0; c < kKeys; ++c) s[c] = c <= lim ? s[c] : -INFINITY;
      }
      float mx = s[0];
#pragma unroll
      for (int c = 1; c < kKeys; ++c) mx = fmaxf(mx, s[c]);
      const float m_old = m;
      m = fmaxf(m, mx * pd.qscale);
      const float mu = m == -INFINITY ? 0.f : m;  // a row with no finite score so far
      const float alpha = ex2(m_old - mu);
      l *= alpha;
      uint32_t p[kKeys / 2];
      float part[4] = {0.f, 0.f, 0.f, 0.f};  // sums of 32 keys
#pragma unroll
      for (int c = 0; c < kKeys; c += 2) {
        const float p0 = ex2(fmaf(s[c], pd.qscale, -mu)), p1 = ex2(fmaf(s[c + 1], pd.qscale, -mu));
        part[c / 32] += p0 + p1;
        p[c / 2] = h2_as_u32(__floats2half2_rn(p0, p1));
      }
      l += (part[0] + part[1]) + (part[2] + part[3]);
      if (MASS && slot >= 0) {
        float* q = scr + static_cast<size_t>(j) * (sub_n + 1) * kRows + row;
        if (T == 32) {
#pragma unroll
          for (int k = 0; k < 4; ++k) q[k * kRows] = part[k];
        } else if (T == 64) {
          q[0] = part[0] + part[1];
          q[kRows] = part[2] + part[3];
        } else {
          q[0] = (part[0] + part[1]) + (part[2] + part[3]);
        }
        q[sub_n * kRows] = mu;
      }
      tmem_st32<0>(tS + tlane, p);
      tmem_st32<32>(tS + tlane + 32, p);
      if (j > 0 && __any_sync(kFull, alpha != 1.f)) {
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32<0>(tO + tlane + c, o);
          tmem_wait32<0>(o);
          uint32_t x[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(o[e] * alpha);
          tmem_st32<0>(tO + tlane + c, x);
        }
      }
      tmem_wait_st();
      fence_before();
      __syncthreads();
      if (tid == 0) {
        fence_after();
        for (int k = 0; k < kKeys / 16; ++k)
          mma_ts(tO, tS + 8 * k, sw128_desc(s0 + Geo::kV + k * 2048, kKeys * 128), idesc_m128(D, true), j > 0 || k > 0);
        mma_commit(bar_mma);
      }
      ok = mbar_wait(bar_mma, ph_mma, stop);
      if (__syncthreads_or(!ok)) {
        failed = true;
        break;
      }
      ph_mma ^= 1;
      fence_after();
    }
    if (failed) break;
    ph_q ^= 1;

    // ---- the unit's rows
    const bool odd = *odd_v != 0;
    const float inv = 1.f / l;
    const size_t orow = (static_cast<size_t>(u.first + (live ? ti : 0)) * nh * G + u.head * G + row % G);
    __half* out = static_cast<__half*>(a.out) + orow * D;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float o[32];
      tmem_ld32<0>(tO + tlane + c, o);
      tmem_wait32<0>(o);
      if (!live) continue;
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] *= inv;
      if (odd) {  // the values left out above, to the rows that see them
        for (int key = edge * kKeys; key <= vis; ++key) {
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
      __syncthreads();
      float* dst = pd.part + static_cast<size_t>(slot) * pd.max_tiles_k * sub_n;
      for (int i = tid; i < nk * sub_n; i += kThreads) {
        const float* ps = scr + (static_cast<size_t>(i / sub_n) * (sub_n + 1) + i % sub_n) * kRows;
        const float* pm = scr + (static_cast<size_t>(i / sub_n) * (sub_n + 1) + sub_n) * kRows;
        float sum = 0.f;
        for (int r = 0; r < kRows; ++r)
          if (s_w[r] != 0.f) sum += ps[r] * ex2(pm[r] - s_m[r]) * s_w[r];
        dst[i] = sum;
      }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (tid == 0) *odd_v = 0;
  }
  if (failed) {
    // copies in flight land before the shared memory is given back
    if (tid == 0) report_error(a.dev_status, KVQ_ERR_DEVICE_TIMEOUT);
    const long long t0 = global_ns();
    while (global_ns() - t0 < kWaitLimitNs && !mbar_try(bar_kv, ph_kv)) {
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 0) tmem_free512(tm);
}

// mass[s][t] += the partial masses of the units of sequence s that reach tile
// t, over heads and runs in order.  A thread per tile.
__global__ void __launch_bounds__(128) prompt_mass_kernel(PromptDev pd) {
  const PromptArgs& a = pd.a;
  const int s = blockIdx.y, t = blockIdx.x * blockDim.x + threadIdx.x;
  const int T = a.cfg.tile_tokens, W = pd.unit_tokens, nh = a.cfg.num_kv_heads;
  Unit u{s, 0, 0, 0, 0};
  u.n = seq_len(a, s, u.first);
  if (t >= (u.n + T - 1) / T || t >= a.max_tiles) return;
  const int w0 = a.mass_window == 0 ? 0 : max(0, u.n - a.mass_window) / W;
  const int r0 = max(w0, t * T / W), r1 = (u.n + W - 1) / W;
  const size_t stride = static_cast<size_t>(pd.max_tiles_k) * (kKeys / T);
  float sum = 0.f;
  for (u.run = r0; u.run < r1; ++u.run)
    for (u.head = 0; u.head < nh; ++u.head) sum += pd.part[static_cast<size_t>(mass_slot(pd, u)) * stride + t];
  a.mass[static_cast<size_t>(s) * a.max_tiles + t] += sum;
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

int unit_tokens(const kvq_config& cfg) { return kRows / cfg.group_size; }

struct PromptSizes {
  long long units;
  int max_tiles_k, window_units, grid;
  size_t scratch_floats, part_floats;
};
PromptSizes prompt_sizes(const kvq_config& cfg, int num_seqs, int total_tokens, int max_seq_tokens, int window,
                         int sms) {
  PromptSizes z;
  const int W = unit_tokens(cfg), sub = kKeys / cfg.tile_tokens;
  z.units = (static_cast<long long>(total_tokens) / W + num_seqs) * cfg.num_kv_heads;
  z.max_tiles_k = (max_seq_tokens + kKeys - 1) / kKeys;
  z.window_units = window == 0 ? 0 : std::min((window - 1) / W + 2, (max_seq_tokens + W - 1) / W);
  z.grid = static_cast<int>(std::min<long long>(z.units, sms));
  z.scratch_floats = static_cast<size_t>(z.grid) * z.max_tiles_k * (sub + 1) * kRows;
  const size_t slots = window == 0 ? static_cast<size_t>(z.units)
                                   : static_cast<size_t>(num_seqs) * z.window_units * cfg.num_kv_heads;
  z.part_floats = slots * z.max_tiles_k * sub;
  return z;
}

template <int D, bool MASS>
cudaError_t launch_prompt(const PromptArgs& a, cudaStream_t s) {
  int dev = 0, sms = 148;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const PromptSizes z = prompt_sizes(a.cfg, a.num_seqs, a.total_tokens, a.max_seq_tokens, a.mass_window, sms);
  const int G = a.cfg.group_size, nh = a.cfg.num_kv_heads;
  CUtensorMap mq, mk, mv;
  if (!make_map(&mq, a.q, D, nh * G, a.total_tokens, a.q_stride, G, kRows / G) ||
      !make_map(&mk, a.k, D, nh, a.total_tokens, a.k_stride, 1, kKeys) ||
      !make_map(&mv, a.v, D, nh, a.total_tokens, a.v_stride, 1, kKeys))
    return cudaErrorInvalidValue;
  PromptDev pd{};
  pd.a = a;
  pd.unit_tokens = unit_tokens(a.cfg);
  pd.units = static_cast<int>(z.units);
  pd.max_tiles_k = z.max_tiles_k;
  pd.window_units = z.window_units;
  pd.qscale = a.softmax_scale * kLog2e;
  pd.scratch = static_cast<float*>(a.workspace);
  pd.part = pd.scratch + z.scratch_floats;
  auto kern = prompt_kernel<D, MASS>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Geom<D>::kSmem);
  if (e != cudaSuccess) return e;
  kern<<<z.grid, kThreads, Geom<D>::kSmem, s>>>(mq, mk, mv, pd);
  e = cudaGetLastError();
  if (e != cudaSuccess || !MASS) return e;
  const int tiles = std::min(a.max_tiles, (a.max_seq_tokens + a.cfg.tile_tokens - 1) / a.cfg.tile_tokens);
  prompt_mass_kernel<<<dim3((tiles + 127) / 128, a.num_seqs), 128, 0, s>>>(pd);
  return cudaGetLastError();
}

}  // namespace

long long prompt_units(const kvq_config& cfg, int num_seqs, int total_tokens) {
  return (static_cast<long long>(total_tokens) / unit_tokens(cfg) + num_seqs) * cfg.num_kv_heads;
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
