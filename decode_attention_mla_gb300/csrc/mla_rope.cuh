// mla_rope.cuh -- a head's 64 rotated elements in eight lanes: what the kernels
// that rotate them share.
#pragma once

#include <cstdint>

#include "device_utils.cuh"

namespace mla {

__device__ __forceinline__ void widen8(const uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}
// Unit u (of 8) of a head's 64 elements: pairs 4u .. 4u + 3.  Interleaved
// pairs are elements 8u .. 8u + 7 (the ones behind rot_dim pass through in
// place).  Half layout: elements 4u .. and half + 4u ..; the pairs behind the
// rotated ones hold the eight copied elements rot_dim + 2 (4u - half) ...
// Element offsets of a unit's two groups of four.
__device__ __forceinline__ void unit_offsets(int u, int half, int interleaved, int& lo, int& hi) {
    if (interleaved) {
        lo = 8 * u;
        hi = 8 * u + 4;
    } else if (4 * u < half) {
        lo = 4 * u;
        hi = half + 4 * u;
    } else {
        lo = 2 * half + 2 * (4 * u - half);
        hi = lo + 4;
    }
}

// The unit's eight elements, in the order of its two groups.
__device__ __forceinline__ void rotate_unit(float (&f)[8], int interleaved, const float (&cs)[4],
                                            const float (&sn)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // (the indices of both layouts are constants: select, do not index)
        const float x = interleaved ? f[2 * i] : f[i], y = interleaved ? f[2 * i + 1] : f[i + 4];
        const float rx = x * cs[i] - y * sn[i], ry = y * cs[i] + x * sn[i];
        if (interleaved) {
            f[2 * i] = rx;
            f[2 * i + 1] = ry;
        } else {
            f[i] = rx;
            f[i + 4] = ry;
        }
    }
}

__device__ __forceinline__ uint4 load_unit(const uint16_t* p, int lo, int hi) {
    const uint2 a = *reinterpret_cast<const uint2*>(p + lo), b = *reinterpret_cast<const uint2*>(p + hi);
    return make_uint4(a.x, a.y, b.x, b.y);
}

// Sine and cosine of pair `lane` at a position, times the amplitude (0 behind the rotated
// pairs): p * turn modulo 2^64 is the exact fraction of a turn.
__device__ __forceinline__ void pair_angle(int pos, const unsigned long long* turns, int half, float amplitude, int lane,
                                           float& s, float& c) {
    s = c = 0.f;
    if (lane < half) {
        const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(pos)) * turns[lane];
        const float x = static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f;   // units of pi
        sincospif(x, &s, &c);
        c *= amplitude;
        s *= amplitude;
    }
}
// Those of unit u's four pairs, from the lanes that have them.
__device__ __forceinline__ void unit_angles(int u, float s, float c, float (&cs)[4], float (&sn)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        cs[i] = __shfl_sync(0xffffffffu, c, 4 * u + i);
        sn[i] = __shfl_sync(0xffffffffu, s, 4 * u + i);
    }
}

}  // namespace mla
