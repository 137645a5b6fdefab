// decode_window.cu -- the sliding-window (16-bit pools) decode kernel instances with up to 8
// query columns (see launch.cuh); more columns run on the tcgen05 kernel.
#include "launch.cuh"

namespace pkv_host {

namespace {

template <typename T, int D>
pa_status dispatch_window(int bs, const pkv::DecodeArgs& a, const CUtensorMap& mk,
                          const CUtensorMap& mv, int grid, cudaStream_t s) {
  switch (bs) {
    case 1: return launch_decode<T, D, 1, 1, pkv::kWindow>(a, mk, mv, grid, s);
    case 8: return launch_decode<T, D, 8, 1, pkv::kWindow>(a, mk, mv, grid, s);
    case 16: return launch_decode<T, D, 16, 1, pkv::kWindow>(a, mk, mv, grid, s);
    case 32: return launch_decode<T, D, 32, 1, pkv::kWindow>(a, mk, mv, grid, s);
  }
  return PA_ERR_UNSUPPORTED;
}

}  // namespace

template <>
pa_status run_decode_mode<pkv::kWindow, false>(bool bf16, int d, int bs, const pkv::DecodeArgs& a,
                                               const CUtensorMap& mk, const CUtensorMap& mv,
                                               int grid, cudaStream_t s) {
  if (a.ncol > 8) return PA_ERR_UNSUPPORTED;
  if (bf16)
    return d == 64 ? dispatch_window<__nv_bfloat16, 64>(bs, a, mk, mv, grid, s)
                   : dispatch_window<__nv_bfloat16, 128>(bs, a, mk, mv, grid, s);
  return d == 64 ? dispatch_window<__half, 64>(bs, a, mk, mv, grid, s)
                 : dispatch_window<__half, 128>(bs, a, mk, mv, grid, s);
}

}  // namespace pkv_host
