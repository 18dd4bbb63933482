// gemm_ragged_bf16_bf16.cu -- the grouped products for bf16 operands and a bf16 C;
// the kernel templates are in gemm_ragged.cuh.
#include "gemm_ragged.cuh"

namespace libgemm {

int launch_ragged_bf16_bf16(RaggedParams& rp, int mode, int cg, bool p_mn, int64_t units,
                     const DeviceInfo& dev, cudaStream_t s) {
    return dispatch_ragged<true, __nv_bfloat16>(rp, mode, cg, p_mn, units, dev, s);
}

}  // namespace libgemm
