// Paged decode attention and the serving step: launches of the kernels in
// kvq_decode_kernel.cuh without masses.
#include "kvq_decode_kernel.cuh"

namespace kvq {

namespace {

// ------------------------------------------------------------------ self-test
// The decode kernel's bounded wait on a barrier that nothing arrives at.
__global__ void selftest_wait_decode_kernel(int32_t* dev_status) {
  __shared__ __align__(8) uint64_t bar;
  mbar_init(&bar, 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  if (!mbar_wait_bounded(&bar, 0)) report_error(dev_status, KVQ_ERR_DEVICE_TIMEOUT);
}

// the fused serving step: no schedule kernel (a fixed grid of num_splits
// units per (sequence, KV head)), one launch
template <int T, int BK, int BV>
cudaError_t launch_step_bits(const DecodeArgs& a, cudaStream_t s, int sms) {
  using Geo = DecodeGeom<T, BK, BV>;
  auto kern = decode_tiles_kernel<T, BK, BV, false>;
  int per_sm = 0;
  cudaError_t e = decode_ctas_per_sm<T, BK, BV, false>(&per_sm);
  if (e != cudaSuccess) return e;
  kern<<<sms * per_sm, Geo::kWarps * 32, Geo::kSmem, s>>>(a);
  return cudaGetLastError();
}

template <int T, int BK, int BV>
struct DecodeLauncher {
  static cudaError_t run(const DecodeArgs& a, cudaStream_t s, int sms) { return launch_decode_bits<T, BK, BV, false>(a, s, sms); }
};
template <int T, int BK, int BV>
struct StepLauncher {
  static cudaError_t run(const DecodeArgs& a, cudaStream_t s, int sms) { return launch_step_bits<T, BK, BV>(a, s, sms); }
};

template <int T>
cudaError_t launch_decode_t(const DecodeArgs& a, cudaStream_t s) {
  return a.step ? dispatch_decode_bits<T, StepLauncher>(a, s, device_sms())
                : dispatch_decode_bits<T, DecodeLauncher>(a, s, device_sms());
}

}  // namespace

size_t decode_workspace_bytes(const kvq_config& cfg, int num_seqs, int num_splits, int num_sms) {
  if (cfg.head_dim != kHeadDim) return generic_decode_workspace_bytes(cfg, num_seqs, num_splits, num_sms);
  const WsLayout wl = ws_layout(num_seqs, cfg.num_kv_heads, cfg.group_size);
  const size_t units = num_splits > 0
                           ? static_cast<size_t>(num_seqs) * cfg.num_kv_heads * num_splits
                           : static_cast<size_t>(units_per_sm(cfg.tile_tokens)) * num_sms +
                                 static_cast<size_t>(num_seqs) * cfg.num_kv_heads;
  return wl.part_off + units * cfg.group_size * kPartFloats * sizeof(float) + units * sizeof(int32_t);
}

cudaError_t launch_selftest_wait_decode(int32_t* dev_status, cudaStream_t s) {
  selftest_wait_decode_kernel<<<1, 1, 0, s>>>(dev_status);
  return cudaGetLastError();
}

cudaError_t launch_append_decode_step(const DecodeArgs& a, cudaStream_t s) { return launch_paged_decode(a, s); }

cudaError_t launch_paged_decode(const DecodeArgs& a, cudaStream_t s) {
  if (a.cfg.head_dim != kHeadDim) return launch_generic_decode(a, s);
  if (a.num_seqs == 0) return cudaSuccess;
  switch (a.cfg.tile_tokens) {
    case 32: return launch_decode_t<32>(a, s);
    case 64: return launch_decode_t<64>(a, s);
    default: return launch_decode_t<128>(a, s);
  }
}

}  // namespace kvq
