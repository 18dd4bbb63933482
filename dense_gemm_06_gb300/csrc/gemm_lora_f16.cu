// gemm_lora_f16.cu -- the two launches of gemm_lora for f16 operands and C; the
// kernel templates are in gemm_ragged.cuh.
#include "gemm_ragged.cuh"

namespace libgemm {

int launch_lora_f16(RaggedParams& rp, int mode, int cg, bool p_mn, int64_t units,
                const DeviceInfo& dev, cudaStream_t s) {
    return dispatch_lora<false, __half>(rp, mode, cg, p_mn, units, dev, s);
}

}  // namespace libgemm
