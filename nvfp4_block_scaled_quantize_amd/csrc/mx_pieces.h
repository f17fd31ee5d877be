// mx_pieces.h -- what the kernels that decode a copy share: 16 bytes of output a lane, and their way out.
#pragma once
#include "mx_common.h"

namespace nvfp4 {

// The decode's piece of a lane: 16 bytes of output, so that a wave's stores are contiguous.
template <typename T> struct Piece;
template <> struct Piece<uint16_t> { static constexpr int n = 8; using Codes = uint32_t; };
template <> struct Piece<float> { static constexpr int n = 4; using Codes = uint16_t; };

// Dword-aligned vectors, stored past the caches: 8192 x 9216 bfloat16 28 us against 38 with
// ordinary stores, and 60 against 66 together with a quantizer that reads them back.
typedef int int3a __attribute__((ext_vector_type(3), aligned(4)));

// Stores the piece d at p, of which `left` elements lie in the row (<= 0: none).  Lanes of a
// wave hold consecutive pieces; `first`: the previous lane's is not the one before this in its
// row.  Where p is an odd bfloat16, the lane stores the dwords that its piece ends, taking the
// previous lane's last element, so that rows of any pitch are written in dwords: 4096 x 8191
// bfloat16 16 us against 22 with 16-byte stores at odd addresses.  All 64 lanes call.
template <typename T>
__device__ __forceinline__ void store_piece(int4v d, T* p, int64_t left, bool first) {
    constexpr int n = Piece<T>::n;
    if constexpr (sizeof(T) == 2) {
        const int before = dpp<kWaveShr1>(0, d[3]);
        if (((uintptr_t)p & 2) && left >= n) {
            const int4v o = {(int)__builtin_amdgcn_alignbit(d[0], before, 16), (int)__builtin_amdgcn_alignbit(d[1], d[0], 16),
                             (int)__builtin_amdgcn_alignbit(d[2], d[1], 16), (int)__builtin_amdgcn_alignbit(d[3], d[2], 16)};
            if (first) {
                *p = (T)d[0];
                __builtin_nontemporal_store((int3a){o[1], o[2], o[3]}, (int3a*)(p + 1));
            } else {
                __builtin_nontemporal_store((int4_by4)o, (int4_by4*)(p - 1));
            }
            // no whole piece after this one in the wave: nobody else stores the last element
            if (left < 2 * n || (threadIdx.x & 63) == 63) p[n - 1] = (T)((uint32_t)d[3] >> 16);
            return;
        }
    }
    if (left >= n) {
        __builtin_nontemporal_store((int4_by4)d, (int4_by4*)p);
        return;
    }
    T e[n];
    __builtin_memcpy(e, &d, sizeof(e));
#pragma unroll
    for (int i = 0; i < n; ++i)
        if (i < left) p[i] = e[i];
}

}  // namespace nvfp4
