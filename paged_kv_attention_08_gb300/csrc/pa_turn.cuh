// Rotary pieces shared by the appends to the 8-bit and the latent cache: a
// table of sines and cosines in shared memory, and the turn of eight pairs.
#pragma once

#include "pa_device.cuh"

namespace pa {

// Sine and cosine of pair j of token t of a CTA at [t][4][octets] float4
// (cos, sin) x 2, octets = pairs / 8: threads of neighbouring octets read
// neighbouring vectors.
__device__ __forceinline__ float2* turn_entry(float4* cs, int octets, int t, int j) {
    return reinterpret_cast<float2*>(cs + (t * 4 + ((j >> 1) & 3)) * octets + (j >> 3)) + (j & 1);
}

// The angle of a position, modulo one turn in 64-bit integers (exact for far
// positions), as (cos, sin) in 32 bits.
__device__ __forceinline__ float2 turn_angle(int32_t position, int64_t phase) {
    const unsigned long long turn = (unsigned long long)(long long)position * (unsigned long long)phase;
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c, s);
}

// Sixteen elements of a head, widened: lo holds elements 0..7 and hi 8..15 of
// the two 8-element vectors that an item of eight pairs loads.
template <typename T>
__device__ __forceinline__ void widen8(const uint4& lo, const uint4& hi, float (&x)[16]) {
    const uint32_t a[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) Mma<T>::unpack(a[i], x[2 * i], x[2 * i + 1]);
}

// Eight pairs turned in place: pair i is (x[i], x[8 + i]), or (x[2i], x[2i + 1])
// interleaved; cs: the item's first vector of the table.
__device__ __forceinline__ void turn8(float (&x)[16], const float4* cs, int octets, bool interleaved) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float4 w = cs[c * octets];
        if (interleaved) {
            const float a0 = x[4 * c], b0 = x[4 * c + 1], a1 = x[4 * c + 2], b1 = x[4 * c + 3];
            x[4 * c] = a0 * w.x - b0 * w.y;
            x[4 * c + 1] = a0 * w.y + b0 * w.x;
            x[4 * c + 2] = a1 * w.z - b1 * w.w;
            x[4 * c + 3] = a1 * w.w + b1 * w.z;
        } else {
            const float a0 = x[2 * c], b0 = x[8 + 2 * c], a1 = x[2 * c + 1], b1 = x[8 + 2 * c + 1];
            x[2 * c] = a0 * w.x - b0 * w.y;
            x[8 + 2 * c] = a0 * w.y + b0 * w.x;
            x[2 * c + 1] = a1 * w.z - b1 * w.w;
            x[8 + 2 * c + 1] = a1 * w.w + b1 * w.z;
        }
    }
}

// Rounded back to 16 bits, each element once.
template <typename T>
__device__ __forceinline__ void narrow8(const float (&x)[16], uint4& lo, uint4& hi) {
    lo = make_uint4(Mma<T>::pack(x[0], x[1]), Mma<T>::pack(x[2], x[3]), Mma<T>::pack(x[4], x[5]),
                    Mma<T>::pack(x[6], x[7]));
    hi = make_uint4(Mma<T>::pack(x[8], x[9]), Mma<T>::pack(x[10], x[11]), Mma<T>::pack(x[12], x[13]),
                    Mma<T>::pack(x[14], x[15]));
}

}  // namespace pa
