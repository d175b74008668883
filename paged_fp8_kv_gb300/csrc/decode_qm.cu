// The query-rows decode kernel on plain scores (see decode_qm.cuh).

#include "decode_qm.cuh"

namespace mj {

cudaError_t launch_decode_qm(const DecodeDev& a, int rows_per_cta, int n_q_tiles, bool q_e4m3, cudaStream_t stream) {
  return launch_qm_rows<false>(a, rows_per_cta, n_q_tiles, q_e4m3, stream);
}

int qm_smem_bytes(bool q_e4m3) { return q_e4m3 ? QmCfg<true>::kBytes : QmCfg<false>::kBytes; }

}  // namespace mj
