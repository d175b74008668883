// The swap-AB decode kernel on modified scores (see decode_tc.cuh): up to 16
// packed rows, where mj_decode_attn takes it too.

#include "decode_tc.cuh"

namespace mj {

cudaError_t launch_decode_tc_mod(const DecodeModDev& a, int rows_per_cta, int n_q_tiles, bool q_e4m3,
                                 cudaStream_t stream) {
  switch (rows_per_cta) {
    case 8:
      return q_e4m3 ? launch_tc<8, true, false, true>(a, n_q_tiles, stream)
                    : launch_tc<8, false, false, true>(a, n_q_tiles, stream);
    case 16:
      return q_e4m3 ? launch_tc<16, true, false, true>(a, n_q_tiles, stream)
                    : launch_tc<16, false, false, true>(a, n_q_tiles, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mj
