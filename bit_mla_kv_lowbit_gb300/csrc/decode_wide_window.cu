// The cluster kernel (decode_wide.cuh) for the windowed decode.
#include "decode_wide.cuh"

namespace mlalb {

template <bool kOne, bool kMixed>
static cudaError_t launch(int cbits, const DecodeArgs& a, cudaStream_t stream) {
  return launch_wide(cbits, a, stream,
                     cbits == 4   ? wide::decode_wide_kernel<4, true, kOne, kMixed>
                     : cbits == 2 ? wide::decode_wide_kernel<2, true, kOne, kMixed>
                                  : wide::decode_wide_kernel<16, true, kOne, kMixed>,
                     true);
}
cudaError_t launch_decode_wide_window(int cbits, const DecodeArgs& a, cudaStream_t stream) {
  const bool one = a.win_cut.splits == 1;
  if (a.n_q > 1 && a.H / a.n_q % wide::kRows != 0)
    return one ? launch<true, true>(cbits, a, stream) : launch<false, true>(cbits, a, stream);
  return one ? launch<true, false>(cbits, a, stream) : launch<false, false>(cbits, a, stream);
}

}  // namespace mlalb
