// mx_tile128.hip -- the plain products on 128 x 128 tiles (kernel: mx_tile128.h).
#include "mx_tile128.h"

namespace nvfp4 {
using namespace tile128;

template <typename T, bool STREAM>
static int launch_mode(const MxGArgs& g, int mode, hipStream_t st) {
    return mode == MxDense ? launch<T, MxDense, STREAM>(g, st)
           : mode == MxRows ? launch<T, MxRows, STREAM>(g, st) : launch<T, MxK, STREAM>(g, st);
}

int mx_tile128(const MxGArgs& g, int mode, int c_dtype, bool stream, hipStream_t st) {
    if (c_dtype == NVFP4_BF16) return launch_mode<uint16_t, true>(g, mode, st);
    return stream ? launch_mode<float, true>(g, mode, st) : launch_mode<float, false>(g, mode, st);
}

}  // namespace nvfp4
