// build-flags: -mllvm -amdgpu-mfma-vgpr-form
// The LDS-tiled gate/up GEMM that also keeps both projections as MXFP8
// checkpoints for the backward pass (tiled_gemm_kernel.h with CKPT): the
// projections never leave the chip in 16 bits, only as codes (1 + 1/32 B a
// value each). Same tile shapes as the inference gate/up.
#include "tiled_gemm_kernel.h"

namespace moe {

MOE_BOUNDS_FILE(tiled_ckpt)

hipError_t launch_tiled_ckpt(const GemmProblem &p, int bm, hipStream_t s) {
    if (p.extra_group >= 0 || p.ksplit != 1 || p.tail_part || p.N % mx8::kGroup ||
        !tiled_gemm_supports(W_BF16, p.N, p.K) || !p.ckpt[0] || !p.ckpt[1] || !p.ckpt[2] || !p.ckpt[3])
        return hipErrorInvalidValue;
    if (bm == 256) return tiled::launch_t<W_BF16, true, 256, 2, false, 4, true>(p, s);
    if (bm == 128) return tiled::launch_t<W_BF16, true, 128, 2, false, 2, true>(p, s);
    return hipErrorInvalidValue;
}

}  // namespace moe
