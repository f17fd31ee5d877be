// mx_ffn_forward256.hip -- the gated feed-forward block's forward on 256 x 256 tiles (kernel: mx_tile256.h).
#include "mx_tile256.h"

namespace nvfp4 {

template <int ACT>
static int launch_mode(const MxFfnArgs& f, int mode, hipStream_t st) {
    return mode == MxDense ? tile256::launch<uint16_t, MxDense, true, kForward, ACT>(f, st)
                           : tile256::launch<uint16_t, MxRows, true, kForward, ACT>(f, st);
}

int mx_forward256(const MxFfnArgs& f, int mode, int act, hipStream_t st) {
    return act == MXFP4_SILU ? launch_mode<MXFP4_SILU>(f, mode, st) : launch_mode<MXFP4_GELU>(f, mode, st);
}

}  // namespace nvfp4
