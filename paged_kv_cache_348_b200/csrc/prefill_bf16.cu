// prefill_bf16.cu -- the bf16 instances of the prompt attention kernel (see launch.cuh).
#include "launch.cuh"
#include "prefill.cuh"

namespace pkv_host {

pa_status run_prefill_bf16(int d, int bs, const pkv::PrefillArgs& a, const CUtensorMap& mk,
                         const CUtensorMap& mv, const CUtensorMap& mq, int grid, cudaStream_t s) {
  return dispatch_prefill<__nv_bfloat16>(d, bs, a, mk, mv, mq, grid, s);
}

}  // namespace pkv_host
