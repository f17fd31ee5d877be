// mx_ffn_forward128.hip -- the gated feed-forward block's forward on 128 x 128 tiles (kernel: mx_tile128.h).
#include "mx_tile128.h"

namespace nvfp4 {

template <typename T, int ACT>
static int launch_mode(const MxFfnArgs& f, int mode, hipStream_t st) {
    return mode == MxDense ? tile128::launch<T, MxDense, sizeof(T) == 2, kForward, ACT>(f, st)
                           : tile128::launch<T, MxRows, sizeof(T) == 2, kForward, ACT>(f, st);
}

int mx_forward128(const MxFfnArgs& f, int mode, int dtype, int act, hipStream_t st) {
    if (act == MXFP4_SILU)
        return dtype == NVFP4_BF16 ? launch_mode<uint16_t, MXFP4_SILU>(f, mode, st) : launch_mode<float, MXFP4_SILU>(f, mode, st);
    return dtype == NVFP4_BF16 ? launch_mode<uint16_t, MXFP4_GELU>(f, mode, st) : launch_mode<float, MXFP4_GELU>(f, mode, st);
}

}  // namespace nvfp4
