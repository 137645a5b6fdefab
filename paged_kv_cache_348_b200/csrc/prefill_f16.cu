// prefill_f16.cu -- the fp16 instances of the prompt attention kernel (see launch.cuh).
#include "launch.cuh"
#include "prefill.cuh"

namespace pkv_host {

pa_status run_prefill_f16(int d, int bs, const pkv::PrefillArgs& a, const CUtensorMap& mk,
                         const CUtensorMap& mv, const CUtensorMap& mq, int grid, cudaStream_t s) {
  return dispatch_prefill<__half>(d, bs, a, mk, mv, mq, grid, s);
}

}  // namespace pkv_host
