// xent_f16.cu -- the logits' kernel of gemm_xent() and gemm_xent_grad() for f16
// operands, every mode and CTA group; the kernel template is in xent.cuh.
#include "xent.cuh"

namespace libgemm {

int launch_xent_f16(XentParams& xp, int mode, int cg, const DeviceInfo& dev, cudaStream_t s) {
    return launch_xent<false>(xp, mode, cg, dev, s);
}

}  // namespace libgemm
