// mx_ffn_backward256.hip -- the gated feed-forward block's backward on 256 x 256 tiles (kernel: mx_tile256.h).
#include "mx_tile256.h"

namespace nvfp4 {

template <typename T, int ACT>
static int launch_mode(const MxFfnArgs& f, int mode, hipStream_t st) {
    return mode == MxDense ? tile256::launch<T, MxDense, sizeof(T) == 2, kBackward, ACT>(f, st)
                           : tile256::launch<T, MxRows, sizeof(T) == 2, kBackward, ACT>(f, st);
}

int mx_backward256(const MxFfnArgs& f, int mode, int dtype, int act, hipStream_t st) {
    if (act == MXFP4_SILU)
        return dtype == NVFP4_BF16 ? launch_mode<uint16_t, MXFP4_SILU>(f, mode, st) : launch_mode<float, MXFP4_SILU>(f, mode, st);
    return dtype == NVFP4_BF16 ? launch_mode<uint16_t, MXFP4_GELU>(f, mode, st) : launch_mode<float, MXFP4_GELU>(f, mode, st);
}

}  // namespace nvfp4
