// gemm_ragged_f16_f32.cu -- the grouped products for f16 operands and a f32 C;
// the kernel templates are in gemm_ragged.cuh.
#include "gemm_ragged.cuh"

namespace libgemm {

int launch_ragged_f16_f32(RaggedParams& rp, int mode, int cg, bool p_mn, int64_t units,
                     const DeviceInfo& dev, cudaStream_t s) {
    return dispatch_ragged<false, float>(rp, mode, cg, p_mn, units, dev, s);
}

}  // namespace libgemm
