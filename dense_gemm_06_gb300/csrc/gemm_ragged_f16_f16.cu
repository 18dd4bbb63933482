// gemm_ragged_f16_f16.cu -- the grouped products for f16 operands and a f16 C;
// the kernel templates are in gemm_ragged.cuh.
#include "gemm_ragged.cuh"

namespace libgemm {

int launch_ragged_f16_f16(RaggedParams& rp, int mode, int cg, bool p_mn, int64_t units,
                     const DeviceInfo& dev, cudaStream_t s) {
    return dispatch_ragged<false, __half>(rp, mode, cg, p_mn, units, dev, s);
}

}  // namespace libgemm
